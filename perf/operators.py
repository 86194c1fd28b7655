"""Timing cases of the serving operators: what one pass reads, computes and returns.

Four operators around the gated block-sparse attention: rotary positions
(`sas_rotary`), block tables and slot maps from request lengths
(`sas_page_map`), the cache write with its block summaries
(`sas_cache_append`) and attention of a tree of drafted tokens over the cache
(`sas_decode_tree`). `own` chooses between their plain torch form and the
library's calls; `exact` states each one a second time, in 64 bits.

The scores of a selection are planted, as everywhere in this repository, so
that the order near the Top-K boundary is decided by far more than rounding.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64
TOPICS = 3  # directions of the planted scores; a drafted token follows one of them


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one sequence of the 64K decode workload checked four drafted tokens deep: the
        # smallest verification step, where launch latency counts
        dict(name="tree_chain_64k", op="tree", dtype="bf16", B=1, Hq=32, Hkv=8, d=128, Lmax=65536,
             lo=65500, hi=65500, T=4, topk=15, tree="chain", ragged=False, paged=False,
             sums="f32", gated=1),
        # the batched decode workload: eight ragged sequences, sixteen drafted tokens each,
        # paged cache with bf16 page summaries
        dict(name="tree_batch8_128k", op="tree", dtype="bf16", B=8, Hq=32, Hkv=8, d=128,
             Lmax=131072, lo=98304, hi=131008, T=16, topk=31, tree="random", ragged=True,
             paged=True, sums="bf16", gated=1),
        # the 512K decode workload with the largest tree
        dict(name="tree_wide_512k", op="tree", dtype="bf16", B=1, Hq=32, Hkv=8, d=128, Lmax=524288,
             lo=524200, hi=524200, T=64, topk=63, tree="random", ragged=False, paged=False,
             sums="f32", gated=1),
        # an odd group, head dimension 64 and fp32 caches, gates left out of the logits
        dict(name="tree_f32_odd", op="tree", dtype="f32", B=3, Hq=6, Hkv=2, d=64, Lmax=4160,
             lo=1000, hi=4100, T=7, topk=5, tree="random", ragged=True, paged=False, sums="f32",
             gated=0),
        # training: q and k of the 16K workload, rotated as they leave a fused projection
        # [B][N][heads][d]
        dict(name="rotary_train_16k", op="rotary", dtype="bf16", B=1, Hq=32, Hkv=8, d=128,
             N=16384, rot=128, interleaved=False, inverse=False, scaling="none", factor=1.0,
             start=0, where="start", projected=True),
        # its backward pass in fp32 on part of an odd-sized head, neighbouring pairs
        dict(name="rotary_bwd_f32_odd", op="rotary", dtype="f32", B=2, Hq=6, Hkv=2, d=64, N=1537,
             rot=48, interleaved=True, inverse=True, scaling="linear", factor=4.0, start=0,
             where="pos", projected=False),
        # the drafted tokens of a tree at 512K, frequencies scaled for the long context
        dict(name="rotary_tree_512k", op="rotary", dtype="bf16", B=1, Hq=32, Hkv=8, d=128, N=64,
             rot=128, interleaved=False, inverse=False, scaling="parts", factor=16.0,
             start=524200, where="tree", projected=False),
        # one decode step of eight sequences: q rotated, k rotated and written, v written
        dict(name="append_decode_b8", op="append", dtype="bf16", B=8, Hq=32, Hkv=8, d=128, T=1,
             lo=2000, hi=4095, extra=64, rot=128, interleaved=False, scaling="none", factor=1.0,
             paged=True, sums="f32", with_q=True, accept=False),
        # chunks of two prompts into a paged cache, page summaries in bf16
        dict(name="append_prompt_8k", op="append", dtype="bf16", B=2, Hq=32, Hkv=8, d=128, T=8192,
             lo=1, hi=3000, extra=8192, rot=128, interleaved=False, scaling="none", factor=1.0,
             paged=True, sums="bf16", with_q=False, accept=False),
        # the accepted paths of drafted trees, already rotated, into a contiguous cache
        dict(name="append_accept_b8", op="append", dtype="bf16", B=8, Hq=32, Hkv=8, d=128, T=16,
             lo=2000, hi=4000, extra=96, rot=0, interleaved=False, scaling="none", factor=1.0,
             paged=False, sums="f32", with_q=False, accept=True),
        # tables of a decode step of 256 requests
        dict(name="pages_decode_b256", op="pages", B=256, T=1, lo=0, hi=131071, nlo=1, full=False),
        # tables of 64 prompts of up to 8192 tokens
        dict(name="pages_prompt_b64", op="pages", B=64, T=8192, lo=0, hi=4096, nlo=0, full=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "rotary", "append", "pages"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "pages":
        hi = _log_int(rng, 1, 131071)
        T = _log_int(rng, 1, 8192)
        B = max(1, min(_log_int(rng, 1, 1024), (64 * 8192) // T))
        return dict(op="pages", B=B, T=T, lo=0, hi=hi, nlo=rng.choice([0, 1]),
                    full=rng.random() < 0.5)
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    if Hq > 32:
        Hq, Hkv = 32, 8
    if op == "rotary":
        where = rng.choice(["start", "pos", "tree"])
        N = rng.randint(1, 64) if where == "tree" else _log_int(rng, 1, 16384)
        B = max(1, min(rng.randint(1, 4), 16384 // N))
        return dict(op="rotary", dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, d=d, N=N,
                    rot=rng.choice([d, d, d // 2, 48, 20]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "base", "parts"]),
                    factor=float(rng.randint(2, 32)),
                    start=_log_int(rng, 1, 524288) if rng.random() < 0.7 else 0, where=where,
                    projected=rng.random() < 0.5)
    if op == "append":
        accept = rng.random() < 0.3
        T = rng.randint(1, 64) if accept else _log_int(rng, 1, 8192)
        B = max(1, min(_log_int(rng, 1, 16), 16384 // T))
        hi = _log_int(rng, 1, 4096)
        return dict(op="append", dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, d=d, T=T, lo=0, hi=hi,
                    extra=T + rng.randint(0, 130), rot=0 if accept else rng.choice([d, d // 2, 20]),
                    interleaved=rng.random() < 0.5, scaling="none", factor=1.0,
                    paged=rng.random() < 0.5, sums=rng.choice(["f32", "bf16"]),
                    with_q=(not accept) and rng.random() < 0.5, accept=accept)
    T = rng.randint(1, 64)
    hi = _log_int(rng, 1, 131072)
    topk = rng.choice([0, 1, 2, 7, 15, 31, 33])
    if dtype == "f32":
        hi, T = min(hi, 16384), min(T, 24)
    # no more attended keys than the batched case has
    B = max(1, min(_log_int(rng, 1, 8), 128 * 32 * 31 // (T * Hq * max(topk, 1))))
    return dict(op="tree", dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, d=d,
                Lmax=BLOCK * (hi // BLOCK + 1 + rng.randint(0, 3)), lo=(3 * hi) // 4, hi=hi, T=T,
                topk=topk, tree=rng.choice(["chain", "random"]),
                ragged=rng.random() < 0.5, paged=rng.random() < 0.5,
                sums=rng.choice(["f32", "bf16"]), gated=rng.choice([0, 1, 1]))


# -------------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _spread(lo, hi, B):
    """B lengths of the case's range, ragged, the same for every seed."""
    return [int(lo + (hi - lo) * ((0.618034 * (b + 1)) % 1.0)) for b in range(B)]


def _frequencies(rot, scaling, factor, base=10000.0, trained=8192):
    """fp32 inverse frequencies and the amplitude of the rotation.

    linear: positions divided by factor; base: the base raised so that the
    slowest pair is slowed by factor; parts: slow pairs slowed by factor, fast
    ones kept, a ramp between them over the number of turns that a pair makes
    in the trained length, and a slightly larger amplitude.
    """
    half = rot // 2
    e = np.arange(half, dtype=np.float64) * 2.0 / rot
    if scaling == "base":
        base = base * factor ** (rot / max(rot - 2, 1))
    f = base ** -e
    amp = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        turns = trained * f / (2.0 * np.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * keep + (f / factor) * (1.0 - keep)
        amp = 0.1 * math.log(factor) + 1.0
    return torch.from_numpy(f.astype(np.float32)), float(np.float32(amp))


def _parents(kind, B, T, g):
    """Parent of each drafted token (-1: the last token of the cache)."""
    if kind == "chain":
        p = torch.arange(T, dtype=torch.int32) - 1
        return p.repeat(B, 1).contiguous()
    p = torch.full((B, T), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(1, T):
            # a tree that is a few tokens wide: usually one of the last three
            back = int(torch.randint(1, 4, (1,), generator=g))
            p[b, i] = i - back if i - back >= 0 else -1
    return p


def _depths(par):
    B, T = par.shape
    dep = torch.zeros((B, T), dtype=torch.int32)
    for b in range(B):
        for i in range(T):
            dep[b, i] = 0 if par[b, i] < 0 else dep[b, int(par[b, i])] + 1
    return dep


def _prepare_tree(c, seed):
    dev = "cuda"
    gc = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, d, T, k = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"], c["topk"]
    G, C = Hq // Hkv, c["Lmax"] // BLOCK
    dt, sdt = _dt(c["dtype"]), _dt(c["sums"])
    lens = _spread(c["lo"], c["hi"], B)
    scale = 1.0 / math.sqrt(d)
    kappa = 6.0
    par = _parents(c["tree"], B, T, gc)
    ntok = [max(1, T - (3 * b) % T) if c["ragged"] else T for b in range(B)]
    topic = torch.randint(0, TOPICS, (B, T), generator=gc)
    pages = torch.randperm(B * C + 3, generator=gc)[:B * C].reshape(B, C).to(torch.int32)
    npages = B * C + 3
    if c["paged"]:
        kc = torch.zeros((npages, Hkv, BLOCK, d), device=dev, dtype=dt)
        vc = torch.zeros_like(kc)
        ksum = torch.zeros((npages, Hkv, d), device=dev, dtype=sdt)
    else:
        kc = torch.empty((B, Hkv, C * BLOCK, d), device=dev, dtype=dt)
        vc = torch.empty_like(kc)
        ksum = torch.empty((B, Hkv, C, d), device=dev, dtype=sdt)
    q = torch.empty((B, Hq, T, d), device=dev, dtype=dt)
    kd = torch.empty((B, Hkv, T, d), device=dev, dtype=dt)
    vd = torch.randn((B, Hkv, T, d), generator=g, device=dev).to(dt)
    for b in range(B):
        w = torch.linalg.qr(torch.randn((Hkv, d, TOPICS), generator=g, device=dev))[0]  # [r][d][e]
        # score levels of each topic: P blocks 0.02 apart above 1, the others below 0.8
        planted = C if C <= 4 * max(k, 1) else 2 * max(k, 1)
        shared = planted if planted == C else (7 * planted) // 10
        level = 0.25 * torch.randn((Hkv, TOPICS, C), generator=g, device=dev)
        level = torch.clamp(level, max=0.8)
        for r in range(Hkv):
            order = torch.randperm(C, generator=gc).to(dev)
            for e in range(TOPICS):
                own_part = order[shared + e * (planted - shared):][:planted - shared]
                chosen = torch.cat([order[:shared], own_part])
                rank = torch.randperm(chosen.numel(), generator=gc).to(dev)
                level[r, e, chosen] = 1.0 + 0.02 * rank.float()
        alpha = level / (scale * kappa)
        mean = torch.einsum("rec,rde->rcd", alpha, w)
        for r in range(Hkv):
            x = torch.randn((C, BLOCK, d), generator=g, device=dev)
            x += (mean[r] - x.mean(1)).unsqueeze(1)
            x = x.to(dt)
            s = x.double().mean(1)
            v = torch.randn((C, BLOCK, d), generator=g, device=dev).to(dt)
            if c["paged"]:
                at = pages[b].long().to(dev)
                kc[at, r], vc[at, r], ksum[at, r] = x, v, s.to(sdt)
            else:
                kc[b, r], vc[b, r], ksum[b, r] = x.reshape(-1, d), v.reshape(-1, d), s.to(sdt)
        # drafted queries along their topic; drafted keys as the cache's, near every topic
        x = torch.randn((Hkv, G, T, d), generator=g, device=dev)
        x -= torch.einsum("rgtd,rde,rfe->rgtf", x, w, w)
        x += kappa * w.permute(0, 2, 1)[:, topic[b].to(dev)].unsqueeze(1)
        q[b] = x.reshape(Hq, T, d).to(dt)
        kd[b] = (torch.randn((Hkv, T, d), generator=g, device=dev)
                 + (0.4 / (scale * kappa)) * w.sum(2).unsqueeze(1)).to(dt)
    return dict(op="tree", q=q, kd=kd, vd=vd, kc=kc, vc=vc, ksum=ksum,
                lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                ntok=torch.tensor(ntok, dtype=torch.int32, device=dev),
                parents=par.to(dev), table=pages.to(dev) if c["paged"] else None, topk=k,
                gated=c["gated"], o=torch.zeros_like(q),
                idx=torch.full((B, Hkv, T, k), -1, dtype=torch.int32, device=dev),
                depth=_depths(par).to(dev), Lmax=C * BLOCK, ntok_host=ntok)


def _prepare_rotary(c, seed):
    dev = "cuda"
    gc = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, d, N = c["B"], c["Hq"], c["Hkv"], c["d"], c["N"]
    dt = _dt(c["dtype"])
    f, amp = _frequencies(c["rot"], c["scaling"], c["factor"])
    if c["projected"]:
        x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g, device=dev).to(dt)
        q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    else:
        q = torch.randn((B, Hq, N, d), generator=g, device=dev).to(dt)
        k = torch.randn((B, Hkv, N, d), generator=g, device=dev).to(dt)
    start = torch.tensor([c["start"] + 13 * b for b in range(B)], dtype=torch.int32)
    par = _parents("random", B, N, gc) if c["where"] == "tree" else None
    if par is not None:
        pos = start[:, None] + _depths(par)
    elif c["where"] == "pos":  # several packed documents in a row
        pos = start[:, None] + torch.arange(N, dtype=torch.int32)[None] % max(1, N // 3)
    else:
        pos = start[:, None] + torch.arange(N, dtype=torch.int32)[None]
    return dict(op="rotary", q=q, k=k, f=f.to(dev), amp=amp, rot=c["rot"],
                interleaved=c["interleaved"], inverse=c["inverse"], where=c["where"],
                start=start.to(dev), parents=None if par is None else par.to(dev),
                pos=pos.to(torch.int32).to(dev))


def _prepare_append(c, seed):
    dev = "cuda"
    gc = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, d, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]
    dt, sdt = _dt(c["dtype"]), _dt(c["sums"])
    lens = _spread(c["lo"], c["hi"], B)
    if c["T"] == 1 and B > 1:
        lens[0] = lens[0] // BLOCK * BLOCK + BLOCK - 1  # one sequence completes a block
    C = (c["hi"] + c["extra"]) // BLOCK + 1
    k = torch.randn((B, Hkv, T, d), generator=g, device=dev).to(dt)
    v = torch.randn((B, Hkv, T, d), generator=g, device=dev).to(dt)
    q = torch.randn((B, Hq, T, d), generator=g, device=dev).to(dt) if c["with_q"] else None
    f, amp = _frequencies(c["rot"], c["scaling"], c["factor"]) if c["rot"] else (None, 1.0)
    rows = None
    if c["accept"]:  # an accepted path: ascending rows of the drafted tokens
        ntok = [1 + (5 * b + T // 2) % T for b in range(B)]
        rows = torch.zeros((B, T), dtype=torch.int32)
        for b in range(B):
            rows[b, :ntok[b]] = torch.sort(torch.randperm(T, generator=gc)[:ntok[b]])[0]
    else:
        ntok = [T - (7 * b) % T if T > 1 else 1 for b in range(B)]
    st = dict(op="append", k=k, v=v, q=q, f=None if f is None else f.to(dev), amp=amp,
              rot=c["rot"], interleaved=c["interleaved"],
              lens=torch.tensor(lens, dtype=torch.int32, device=dev),
              ntok=torch.tensor(ntok, dtype=torch.int32, device=dev),
              lens_host=lens, ntok_host=ntok,
              rows=None if rows is None else rows.to(dev), slots=None, C=C)
    if c["paged"]:
        npages = B * C + 2
        pages = torch.randperm(npages, generator=gc)[:B * C].reshape(B, C)
        slots = torch.full((B, T), -1, dtype=torch.int32)
        for b in range(B):
            p = lens[b] + torch.arange(ntok[b])
            slots[b, :ntok[b]] = (pages[b][p // BLOCK] * BLOCK + p % BLOCK).to(torch.int32)
        shape, sshape = (npages, Hkv, BLOCK, d), (npages, Hkv, d)
        st["slots"] = slots.to(dev)
    else:
        shape, sshape = (B, Hkv, C * BLOCK, d), (B, Hkv, C, d)
    st["kc"] = torch.randn(shape, generator=g, device=dev).to(dt)
    st["vc"] = torch.randn(shape, generator=g, device=dev).to(dt)
    st["ksum"] = torch.randn(sshape, generator=g, device=dev).to(sdt)
    return st


def _prepare_pages(c, seed):
    dev = "cuda"
    g = torch.Generator().manual_seed(seed)
    B, T = c["B"], c["T"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g)
    nnew = torch.randint(c["nlo"], T + 1, (B,), generator=g)
    width = (c["hi"] + T + BLOCK - 1) // BLOCK + 1
    have = (lens + BLOCK - 1) // BLOCK
    need = (lens + nnew + BLOCK - 1) // BLOCK - have
    npages = int(have.sum() + need.sum()) + 16
    perm = torch.randperm(npages, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        n = int(have[b])
        table[b, :n] = perm[at:at + n]
        at += n
    free = perm[at:]
    if c["full"] and int(need.sum()) > 0:  # a pool that runs out under the last requests
        free = free[:max(1, int(0.95 * int(need.sum())))]
    return dict(op="pages", lens=lens.to(torch.int32).to(dev), nnew=nnew.to(torch.int32).to(dev),
                table=table.to(dev), free=free.contiguous().to(dev),
                head=torch.zeros(1, dtype=torch.int32, device=dev), T=T, npages=npages)


def prepare(case, seed):
    return dict(tree=_prepare_tree, rotary=_prepare_rotary, append=_prepare_append,
                pages=_prepare_pages)[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def _rotate(x, pos, f, amp, rot, interleaved, inverse):
    """x [B][H][N][d] rotated at pos [B][N]; angles in 64 bits, products in 32."""
    a = pos.double()[:, None, :, None] * f.double()
    c, s = (a.cos() * amp).float(), (a.sin() * (-amp if inverse else amp)).float()
    y = x.float().clone(memory_format=torch.contiguous_format)
    if interleaved:
        x0, x1 = x[..., 0:rot:2].float(), x[..., 1:rot:2].float()
        y[..., 0:rot:2], y[..., 1:rot:2] = x0 * c - x1 * s, x1 * c + x0 * s
    else:
        x0, x1 = x[..., :rot // 2].float(), x[..., rot // 2:rot].float()
        y[..., :rot // 2], y[..., rot // 2:rot] = x0 * c - x1 * s, x1 * c + x0 * s
    return y.to(x.dtype)


def _plain_append(st):
    k, v, kc, vc, ksum = st["k"], st["v"], st["kc"], st["vc"], st["ksum"]
    B, Hkv, T, d = k.shape
    j = torch.arange(T, device=k.device)
    if st["rows"] is not None:
        r = st["rows"].long()[:, None, :, None].expand(B, Hkv, T, d)
        k, v = k.gather(2, r), v.gather(2, r)
    pos = st["lens"].long()[:, None] + j
    qo = None
    if st["rot"]:
        k = _rotate(k, pos, st["f"], st["amp"], st["rot"], st["interleaved"], False)
        if st["q"] is not None:
            qo = _rotate(st["q"], pos, st["f"], st["amp"], st["rot"], st["interleaved"], False)
    for b in range(B):
        n0, n = st["lens_host"][b], st["ntok_host"][b]
        first, last = n0 // BLOCK, (n0 + n) // BLOCK  # blocks first .. last - 1 become complete
        if st["slots"] is not None:
            s = st["slots"][b, :n].long()
            kc[s // BLOCK, :, s % BLOCK] = k[b, :, :n].transpose(0, 1)
            vc[s // BLOCK, :, s % BLOCK] = v[b, :, :n].transpose(0, 1)
            page = s[BLOCK * (first + 1) - 1 - n0::BLOCK] // BLOCK
            ksum[page] = (kc[page].float().sum(2) / BLOCK).to(ksum.dtype)
        else:
            kc[b, :, n0:n0 + n], vc[b, :, n0:n0 + n] = k[b, :, :n], v[b, :, :n]
            blocks = kc[b].unflatten(1, (-1, BLOCK))[:, first:last]
            ksum[b, :, first:last] = (blocks.float().sum(2) / BLOCK).to(ksum.dtype)
    return [kc, vc, ksum] + ([] if qo is None else [qo])


def _plain_pages(st):
    lens, nnew, table, free = st["lens"].long(), st["nnew"].long(), st["table"], st["free"]
    B, width = table.shape
    T, dev = st["T"], lens.device
    end = lens + nnew
    have = (lens + BLOCK - 1) // BLOCK
    need = (end + BLOCK - 1) // BLOCK - have
    fits = (nnew >= 0) & (nnew <= T) & (lens >= 0) & (end <= BLOCK * width)
    need = torch.where(fits, need, torch.zeros_like(need))
    incl = torch.cumsum(need, 0)
    head = st["head"].long()
    ok = fits & ((need == 0) | (head + incl <= free.numel()))
    first = head + incl - need
    i = torch.arange(width, device=dev) - have[:, None]
    fresh = (i >= 0) & (i < need[:, None]) & ok[:, None]
    page = free[(first[:, None] + i).clamp(0, free.numel() - 1)]
    table.copy_(torch.where(fresh, page, table))
    j = torch.arange(T, device=dev)
    pos = lens[:, None] + j
    live = (j < nnew[:, None]) & ok[:, None]
    page = table.long().gather(1, torch.clamp(pos // BLOCK, 0, width - 1))
    slots = torch.where(live, page * BLOCK + pos % BLOCK, torch.full_like(pos, -1))
    granted = torch.where(ok, need, torch.zeros_like(need))
    return [slots.to(torch.int32), torch.where(ok, end, lens).to(torch.int32),
            torch.where(ok, need, torch.full_like(need, -1)).to(torch.int32),
            (head + granted.sum()).to(torch.int32), table]


def _plain_tree(st):
    q, kd, vd, k = st["q"], st["kd"], st["vd"], st["topk"]
    B, Hq, T, d = q.shape
    Hkv = kd.shape[1]
    G, C = Hq // Hkv, st["Lmax"] // BLOCK
    dev = q.device
    scale = 1.0 / math.sqrt(d)
    o, idx_out = st["o"], st["idx"]
    # ancestors (self included) of every token, [B][T][T]
    anc = torch.eye(T, dtype=torch.bool, device=dev).repeat(B, 1, 1)
    hop = st["parents"].long()
    for _ in range(T):
        anc |= (hop[:, :, None] == torch.arange(T, device=dev)) & (hop[:, :, None] >= 0)
        hop = torch.where(hop >= 0, st["parents"].long().gather(1, hop.clamp(min=0)), hop)
    depth = st["depth"].long()
    qg = q.view(B, Hkv, G, T, d)
    qbar = qg.double().mean(2)
    hist = st["lens"].long() // BLOCK  # complete blocks of the cache
    m = torch.arange(C, device=dev)
    for b in range(B):
        at = None if st["table"] is None else st["table"][b].long()
        ks = st["ksum"][b] if at is None else st["ksum"][at].transpose(0, 1)
        s = torch.einsum("rtd,rcd->rtc", qbar[b], ks.double()) * scale
        full = hist[b]
        s = torch.where(m < full, s, torch.full_like(s, -math.inf))
        # the block of the cache's tail, once a path has completed it
        tail = st["lens"].long()[b] - BLOCK * full
        row = BLOCK * full + torch.arange(BLOCK, device=dev)
        in_tail = torch.arange(BLOCK, device=dev) < tail
        row = row.clamp(max=C * BLOCK - 1)
        if at is None:
            kt, vt = st["kc"][b][:, row], st["vc"][b][:, row]
        else:
            page = at[row // BLOCK].clamp(min=0)
            kt, vt = st["kc"][page, :, row % BLOCK].transpose(0, 1), \
                st["vc"][page, :, row % BLOCK].transpose(0, 1)
        zero = torch.zeros((), dtype=kt.dtype, device=dev)
        kt = torch.where(in_tail[:, None], kt, zero)
        vt = torch.where(in_tail[:, None], vt, zero)
        crossed = depth[b] + tail >= BLOCK  # [T]
        early = anc[b] & (depth[b] + tail < BLOCK)[None]  # path keys inside the tail's block
        late = anc[b] & ~early
        mean = (kt.double().sum(1)[:, None] + torch.einsum("tj,rjd->rtd", early.double(),
                                                           kd[b].double())) / BLOCK
        mean = mean.to(st["ksum"].dtype).double()
        sv = (qbar[b] * mean).sum(-1) * scale
        sv = torch.where(crossed, sv, torch.full_like(sv, -math.inf))
        at_full = m == full  # column of the tail's block
        s = torch.cat([torch.where(at_full, sv[..., None], s),
                       torch.where(full >= C, sv, torch.full_like(sv, -math.inf))[..., None]], 2)
        top = s.max(2, keepdim=True)[0]
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        lse = torch.log(torch.exp(s - top).sum(2)) + top[..., 0]
        order = torch.sort(s, dim=2, descending=True, stable=True)[1][..., :k]
        count = torch.minimum(full + crossed.long(), torch.full_like(full, k))  # [T]
        if order.shape[2] < k:
            order = torch.nn.functional.pad(order, (0, k - order.shape[2]), value=C)
        keep = torch.arange(k, device=dev)[None, None] < count[None, :, None]
        kept = torch.sort(torch.where(keep, order, torch.full_like(order, 1 << 30)), dim=2)[0]
        keep = (torch.arange(k, device=dev)[None, None] < count[None, :, None]).expand_as(kept)
        sel = torch.where(keep, kept, torch.full_like(kept, -1))
        logg = torch.where(keep, s.gather(2, kept.clamp(max=C)) - lse[..., None],
                           torch.zeros_like(s[..., :1])).float()
        if st["gated"] == 0:
            logg = torch.zeros_like(logg)
        n = st["ntok_host"][b]
        is_tail = keep & (sel == full)
        tail_bias = torch.where(is_tail.any(2), (logg * is_tail).sum(2),
                                torch.full_like(logg[..., 0], -math.inf)) if k else \
            torch.full((Hkv, T), -math.inf, device=dev)
        tail_bias = torch.where(crossed, tail_bias, torch.zeros_like(tail_bias))  # [r][T]
        for r in range(Hkv):
            qr = qg[b, r].float() * scale  # [G][T][d]
            parts, values = [], []
            if k:
                hm = keep[r] & (sel[r] < full)
                blk = torch.where(hm, sel[r], torch.zeros_like(sel[r])).clamp(max=C - 1)
                if at is None:
                    kb = st["kc"][b, r].view(C, BLOCK, d)[blk]  # [T][k][64][d]
                    vb = st["vc"][b, r].view(C, BLOCK, d)[blk]
                else:
                    kb, vb = st["kc"][at[blk].clamp(min=0), r], st["vc"][at[blk].clamp(min=0), r]
                z = torch.einsum("gtd,tknd->gtkn", qr, kb.float())
                bias = torch.where(hm, logg[r], torch.full_like(logg[r], -math.inf))
                parts.append((z + bias[None, :, :, None]).reshape(G, T, -1))
                values.append(vb.float().reshape(T, -1, d))
            z = torch.einsum("gtd,nd->gtn", qr, kt[r].float())
            z = z + tail_bias[r][None, :, None]
            parts.append(torch.where(in_tail[None, None], z, torch.full_like(z, -math.inf)))
            z = torch.einsum("gtd,jd->gtj", qr, kd[b, r].float())
            bias = torch.where(early, tail_bias[r][:, None].expand(T, T),
                               torch.where(late, 0.0, -math.inf))
            parts.append(z + bias[None])
            z = torch.cat(parts, 2)
            p = torch.exp(z - z.max(2, keepdim=True)[0])
            p = p / p.sum(2, keepdim=True)
            out = torch.einsum("gtn,nd->gtd", p[..., -T - BLOCK:-T], vt[r].float()) \
                + torch.einsum("gtj,jd->gtd", p[..., -T:], vd[b, r].float())
            if k:
                out = out + torch.einsum("gtn,tnd->gtd", p[..., :-T - BLOCK], values[0])
            o[b, r * G:(r + 1) * G, :n] = out[:, :n].to(o.dtype)
        idx_out[b, :, :n] = sel[:, :n].to(torch.int32)
    return [o, idx_out]


def run(state):
    st = state
    if not own:
        if st["op"] == "tree":
            return _plain_tree(st)
        if st["op"] == "rotary":
            a = (st["pos"], st["f"], st["amp"], st["rot"], st["interleaved"], st["inverse"])
            return [_rotate(st["q"], *a), _rotate(st["k"], *a)]
        return _plain_append(st) if st["op"] == "append" else _plain_pages(st)
    from gated_block_sparse_b200 import sas
    if st["op"] == "tree":
        o = sas.sas_decode_tree(st["q"], st["kd"], st["vd"], st["kc"], st["vc"], st["lens"],
                                st["ksum"], st["topk"], parents=st["parents"], ntok=st["ntok"],
                                block_table=st["table"], gated=st["gated"], out=st["o"],
                                idx_out=st["idx"])
        return [o, st["idx"]]
    if st["op"] == "rotary":
        at = dict(pos=st["pos"]) if st["where"] == "pos" else \
            dict(start=st["start"], parents=st["parents"])
        return list(sas.sas_rotary(st["q"], st["f"], k=st["k"], interleaved=st["interleaved"],
                                   amplitude=st["amp"], inverse=st["inverse"], **at))
    if st["op"] == "append":
        qo = sas.sas_cache_append(st["k"], st["v"], st["lens"], st["kc"], st["vc"],
                                  ksum=st["ksum"], ntok=st["ntok"], rows=st["rows"],
                                  slots=st["slots"], inv_freq=st["f"],
                                  interleaved=st["interleaved"], amplitude=st["amp"], q=st["q"])
        return [st["kc"], st["vc"], st["ksum"]] + ([] if qo is None else [qo])
    slots, lens, taken, head = sas.sas_page_map(st["lens"], st["nnew"], st["table"], st["free"],
                                                st["head"], st["T"], st["npages"])
    return [slots, lens, taken, head, st["table"]]


# ------------------------------------------------------------- least work
def work(case):
    c = case
    if c["op"] == "pages":
        # lengths, table entries of the sequences' new pages, slots
        b = 4 * (2 * c["B"] + 2 * c["B"] + c["B"] * c["T"])
        b += 8 * c["B"] * (c["T"] // BLOCK + 1)
        return dict(bytes=b, flops=4 * c["B"] * c["T"])
    es = 2 if c["dtype"] == "bf16" else 4
    d = c["d"]
    if c["op"] == "rotary":
        x = c["B"] * (c["Hq"] + c["Hkv"]) * c["N"]
        return dict(bytes=2 * x * d * es + 4 * c["B"] * c["N"], flops=3 * x * c["rot"])
    ses = 2 if c["sums"] == "bf16" else 4
    if c["op"] == "append":
        T = c["T"]
        if c["accept"]:
            n = sum(1 + (5 * b + T // 2) % T for b in range(c["B"]))
        else:
            n = sum(T - (7 * b) % T if T > 1 else 1 for b in range(c["B"]))
        x = n * c["Hkv"] * d
        b = 4 * x * es + (n // BLOCK) * c["Hkv"] * d * ses
        f = 3 * n * c["Hkv"] * c["rot"] + x
        if c["with_q"]:
            xq = c["B"] * T * c["Hq"]
            b += 2 * xq * d * es
            f += 3 * xq * c["rot"]
        return dict(bytes=b, flops=f)
    B, T, k, Hkv = c["B"], c["T"], c["topk"], c["Hkv"]
    bytes_, flops = 0, 0
    for b, n in enumerate(_spread(c["lo"], c["hi"], B)):
        C, tail = n // BLOCK, n % BLOCK
        t = max(1, T - (3 * b) % T) if c["ragged"] else T
        kk = min(k, C)
        # every summary, one Top-K set and the tail once, the drafted tokens, q and o
        bytes_ += Hkv * (C * d * ses * (k > 0) + (kk * BLOCK + tail + t) * d * es * 2 + 4 * t * k)
        bytes_ += 2 * c["Hq"] * t * d * es
        flops += Hkv * 2 * t * C * d * (k > 0) + c["Hq"] * t * 4 * d * (kk * BLOCK + tail)
    return dict(bytes=bytes_, flops=flops)


# ----------------------------------------------------------------- 64 bits
def _turn(x, pos, st, inverse):
    """The rotation as a product of complex numbers, 64 bits."""
    rot = st["rot"]
    sign = -1.0 if inverse else 1.0
    angle = sign * torch.outer(pos.double().reshape(-1), st["f"].double())
    unit = torch.polar(torch.full_like(angle, st["amp"]), angle).reshape(*pos.shape, rot // 2)
    x = x.double()
    if st["interleaved"]:
        pair = torch.complex(x[..., :rot].unflatten(-1, (rot // 2, 2))[..., 0].contiguous(),
                             x[..., :rot].unflatten(-1, (rot // 2, 2))[..., 1].contiguous())
    else:
        pair = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
    y = pair * unit[:, None]
    if st["interleaved"]:
        head = torch.stack([y.real, y.imag], -1).flatten(-2)
    else:
        head = torch.cat([y.real, y.imag], -1)
    return torch.cat([head, x[..., rot:]], -1)


def _exact_append(st):
    kc, vc, ksum = st["kc"].double(), st["vc"].double(), st["ksum"].double()
    dt = st["k"].dtype
    B, Hkv, T, d = st["k"].shape
    lens, ntok = st["lens_host"], st["ntok_host"]
    j = torch.arange(T, device=kc.device)
    pos = st["lens"].long()[:, None] + j
    k = _turn(st["k"], pos, st, False) if st["rot"] else st["k"].double()
    v = st["v"].double()
    for b in range(B):
        n = ntok[b]
        src = st["rows"][b, :n].long() if st["rows"] is not None else j[:n]
        kb, vb = k[b, :, src], v[b, :, src]
        for blk in range(lens[b] // BLOCK, (lens[b] + n + BLOCK - 1) // BLOCK):
            lo, hi = max(lens[b], BLOCK * blk), min(lens[b] + n, BLOCK * (blk + 1))
            if lo >= hi:
                continue
            a, z = lo - BLOCK * blk, hi - BLOCK * blk
            if st["slots"] is not None:
                page = int(st["slots_host"][b][lo - lens[b]]) // BLOCK
                kd, vd, sd = kc[page], vc[page], ksum[page]
            else:
                kd = kc[b, :, BLOCK * blk:BLOCK * (blk + 1)]
                vd = vc[b, :, BLOCK * blk:BLOCK * (blk + 1)]
                sd = ksum[b, :, blk]
            kd[:, a:z] = kb[:, lo - lens[b]:hi - lens[b]]
            vd[:, a:z] = vb[:, lo - lens[b]:hi - lens[b]]
            if z == BLOCK:  # the mean is that of the stored keys
                sd[...] = kd.to(dt).double().mean(1)
    out = [kc, vc, ksum]
    if st["rot"] and st["q"] is not None:
        out.append(_turn(st["q"], pos, st, False))
    return out


def _exact_tree(st):
    q, kd, vd = st["q"].double(), st["kd"].double(), st["vd"].double()
    B, Hq, T, d = q.shape
    Hkv, k = kd.shape[1], st["topk"]
    G = Hq // Hkv
    dev = q.device
    par, ntok, lens = st["parents"].tolist(), st["ntok"].tolist(), st["lens"].tolist()
    o = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    idx = torch.full((B, Hkv, T, k), -1, dtype=torch.int32, device=dev)
    scale = 1.0 / math.sqrt(d)
    for b in range(B):
        table = None if st["table"] is None else st["table"][b].long()
        n0 = lens[b]
        C0, tail = n0 // BLOCK, n0 % BLOCK

        def block(store, blocks):  # rows of logical blocks, [r][len(blocks)][64][d]
            if table is None:
                return store[b].unflatten(1, (-1, BLOCK))[:, blocks]
            return store[table[blocks]].transpose(0, 1)
        sums = (st["ksum"][b][:, :C0] if table is None
                else st["ksum"][table[:C0]].transpose(0, 1)).double()
        last = torch.tensor([C0], device=dev)
        if tail:
            kt, vt = (block(st[n], last)[:, 0, :tail].double() for n in ("kc", "vc"))
        else:
            kt = vt = torch.zeros((Hkv, 0, d), dtype=torch.float64, device=dev)
        for i in range(ntok[b]):
            path = [i]
            while par[b][path[0]] >= 0:
                path.insert(0, par[b][path[0]])
            # the sequence from the last complete block of the cache on, path appended
            kk = torch.cat([kt, kd[b][:, path]], 1)
            vv = torch.cat([vt, vd[b][:, path]], 1)
            C = (n0 + len(path) - 1) // BLOCK  # history blocks of this token
            summ = sums
            if C > C0:
                new = kk[:, :BLOCK].mean(1, keepdim=True).to(st["ksum"].dtype).double()
                summ = torch.cat([sums, new], 1)
            qi = q[b, :, i].view(Hkv, G, d)
            s = (summ @ qi.mean(1).unsqueeze(-1)).squeeze(-1) * scale  # [r][C]
            gate = torch.log_softmax(s, 1) if C else s
            keep = min(k, C)
            pick = torch.argsort(s, dim=1, descending=True, stable=True)[:, :keep].sort(1)[0]
            idx[b, :, i, :keep] = pick.to(torch.int32)
            ch = BLOCK * (C - C0)  # keys of this stretch that belong to a history block
            z = [torch.einsum("rgd,rnd->rgn", qi, kk[:, ch:]) * scale]
            val = [vv[:, ch:]]
            if keep:
                kb = torch.zeros((Hkv, keep, BLOCK, d), dtype=torch.float64, device=dev)
                vb = torch.zeros_like(kb)
                old = pick < C0
                where = pick.clamp(max=max(C0 - 1, 0))
                if C0:
                    r = torch.arange(Hkv, device=dev)[:, None].expand_as(where)
                    if table is None:
                        kb = st["kc"][b].unflatten(1, (-1, BLOCK))[r, where].double()
                        vb = st["vc"][b].unflatten(1, (-1, BLOCK))[r, where].double()
                    else:
                        kb = st["kc"][table[where], r].double()
                        vb = st["vc"][table[where], r].double()
                if C > C0:
                    kb = torch.where(old[..., None, None], kb, kk[:, None, :BLOCK])
                    vb = torch.where(old[..., None, None], vb, vv[:, None, :BLOCK])
                bias = gate.gather(1, pick) * float(st["gated"])
                zz = torch.einsum("rgd,rknd->rgkn", qi, kb) * scale + bias[:, None, :, None]
                z.append(zz.flatten(2))
                val.append(vb.flatten(1, 2))
            p = torch.softmax(torch.cat(z, 2), 2)
            o[b, :, i] = torch.einsum("rgn,rnd->rgd", p, torch.cat(val, 1)).reshape(Hq, d)
    return [o, idx]


def _exact_pages(st):
    lens, nnew = st["lens"].tolist(), st["nnew"].tolist()
    table, free = st["table"].cpu().numpy().copy(), st["free"].cpu().numpy()
    B, width = table.shape
    T = st["T"]
    head0 = head = int(st["head"].item())
    slots = np.full((B, T), -1, dtype=np.int32)
    out_lens, taken = list(lens), [-1] * B
    want = head0
    for b in range(B):
        n = nnew[b]
        if n < 0 or n > T or lens[b] < 0 or lens[b] + n > BLOCK * width:
            continue
        have = -(-lens[b] // BLOCK)
        need = -(-(lens[b] + n) // BLOCK) - have
        want += need
        if need and want > len(free):
            continue
        table[b, have:have + need] = free[want - need:want]
        head += need
        p = np.arange(lens[b], lens[b] + n)
        slots[b, :n] = table[b, p // BLOCK] * BLOCK + p % BLOCK
        out_lens[b], taken[b] = lens[b] + n, need
    dev = st["lens"].device
    return [torch.from_numpy(slots).to(dev),
            torch.tensor(out_lens, dtype=torch.int32, device=dev),
            torch.tensor(taken, dtype=torch.int32, device=dev),
            torch.tensor([head], dtype=torch.int32, device=dev), torch.from_numpy(table).to(dev)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(st)
    if case["op"] == "append":
        if st["slots"] is not None:
            st["slots_host"] = st["slots"].tolist()
        return _exact_append(st)
    if case["op"] == "pages":
        return _exact_pages(st)
    return [_turn(st["q"], st["pos"], st, st["inverse"]),
            _turn(st["k"], st["pos"], st, st["inverse"])]
