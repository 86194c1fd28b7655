"""The serving calls at sizes that fill the GPU several times: the branches that
only large calls take (several heads or tiles of a CTA, batches of heads, more
CTAs than one wave), against 64-bit arithmetic on the GPU or the oracle.

The tolerances are those of test_gpu_serving.py.
"""
import numpy as np
import pytest
import torch

import serving_cases as S
import test_gpu_serving as T
from gated_block_sparse_b200 import rope, sas
from test_gpu_serving import DEV, HALF, U, clean_status, i32  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def rotated64(x, pos, f, inter, amp):
    """x [B][H][N][d] rotated at pos [B][N] in fp64, on x's device."""
    th = pos.double()[:, None, :, None] * f.double()
    c, s = amp * th.cos(), amp * th.sin()
    y, r = x.double().clone(), 2 * f.numel()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    x0, x1 = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = x0 * c - x1 * s, x1 * c + x0 * s
    pair = torch.zeros_like(y)
    pair[..., a] = pair[..., b] = x0.abs() + x1.abs()
    return y, pair


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("c", [  # dtype, B, N, Hq, Hkv, d, rot, interleaved
    ("bf16", 2, 9700, 7, 3, 128, 128, False), ("bf16", 3, 9700, 5, 1, 64, 32, True),
    ("f32", 2, 4900, 9, 2, 128, 64, True), ("bf16", 2, 1300, 6, 5, 128, 20, False)])
def test_rotary_of_many_tokens(c, inplace):
    """Enough tokens that a thread takes eight heads in two batches, some of q
    and some of k, and head counts that neither divides; fused projections."""
    dtype, B, N, Hq, Hkv, d, rot, inter = c
    f = rope.inv_freq(rot)[0].to(DEV)
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn((B, N, Hq + Hkv, d), generator=g, device=DEV).to(S.TORCH[dtype])
    y = x.clone()
    q, k = (t.transpose(1, 2) for t in (y[:, :, :Hq], y[:, :, Hq:]))
    start = i32([1000 * b for b in range(B)])
    got = sas.sas_rotary(q, f, k=k, start=start, interleaved=inter, out=(q, k) if inplace else None)
    pos = start[:, None] + torch.arange(N, device=DEV)
    for o, t in zip(got, (x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2))):
        ref, pair = rotated64(t, pos, f, inter, 1.0)
        assert torch.equal(o[..., rot:], t[..., rot:])
        tol = pair * 2.0 ** -22.3 + HALF[dtype] * ref.abs()
        assert ((o.double() - ref).abs() <= tol)[..., :rot].all()


@pytest.mark.parametrize("c", [
    # a CTA takes every head: its keys' heads one after the other, then its queries'
    ("bf16", "bf16", 40, 4, 2, 200, 64, [(37 * b) % 190 for b in range(40)],
     [(61 * b) % 201 for b in range(40)], True, 64, False, False, True),
    ("f32", "f32", 40, 3, 3, 200, 128, [(29 * b) % 190 for b in range(40)],
     [200 - (53 * b) % 201 for b in range(40)], False, 128, True, False, True),
    ("bf16", "f32", 38, 2, 2, 200, 64, [(41 * b) % 190 for b in range(38)],
     [(47 * b) % 201 for b in range(38)], True, 20, False, False, True),  # single elements
    ("bf16", "bf16", 50, 6, 6, 150, 64, [(31 * b) % 100 for b in range(50)],
     [(59 * b) % 151 for b in range(50)], True, 0, False, True, False),
    # three heads a CTA, which do not divide the 25
    ("bf16", "f32", 20, 20, 5, 200, 64, [(43 * b) % 190 for b in range(20)],
     [(67 * b) % 201 for b in range(20)], True, 64, True, False, True),
])
def test_cache_append_of_many_tokens(c):
    T.test_cache_append_matches_the_oracle(c)


@pytest.mark.parametrize("dtype,sums,d,paged", [
    ("bf16", "bf16", 128, True), ("bf16", "f32", 64, True), ("bf16", "f32", 128, True),
    ("f32", "bf16", 64, True), ("bf16", "f32", 128, False)])
def test_decode_tree_of_many_groups(dtype, sums, d, paged):
    """Groups enough that a CTA of the scores takes several tiles of summaries,
    in every form of its loop. Queries and summaries are small integers, so
    every score is exact and the selection has to be, ties included; lengths
    end inside the first, second and third tile. Sequences share pages."""
    B, Hq, Hkv, N, C, topk, npages = 64, 16, 8, 33, 300, 21, 330
    G, rng = Hq // Hkv, np.random.Generator(np.random.PCG64(d + len(sums)))
    gen = torch.Generator(device=DEV).manual_seed(d)
    if not paged:
        B, npages = 16, 16 * C  # each sequence has its own
        Hq, Hkv, G = 24, 12, 2
    dt = S.TORCH[dtype]
    draw = lambda lo, hi, shape: torch.randint(lo, hi + 1, shape, generator=gen, device=DEV)
    ksp = draw(-120, 120, (npages, Hkv, d)).to(S.TORCH[sums])
    kp, vp = (torch.randn((npages, Hkv, 64, d), generator=gen, device=DEV).to(dt) for _ in range(2))
    q = draw(-2, 2, (B, Hq, N, d)).to(dt)
    kd, vd = (torch.randn((B, Hkv, N, d), generator=gen, device=DEV).to(dt) for _ in range(2))
    pages = np.stack([rng.permutation(npages)[:C] for _ in range(B)]) if paged else \
        np.arange(B * C).reshape(B, C)
    table = i32(pages)
    lens = [int(64 * C * (0.2 + 0.79 * ((0.618034 * b) % 1.0))) // 64 * 64 + 5 for b in range(B)]
    ntok = [N - (5 * b) % N for b in range(B)]
    scale = 2.0 ** -9
    idx = torch.full((B, Hkv, N, topk), -7, dtype=torch.int32, device=DEV)
    out = torch.full((B, Hq, N, d), 3.0, dtype=dt, device=DEV)
    opt = dict(ntok=i32(ntok), scale=scale, out=out, idx_out=idx)
    if paged:
        sas.sas_decode_tree(q, kd, vd, kp, vp, i32(lens), ksp, topk, block_table=table, **opt)
    else:
        kc, vc = (t.view(B, C, Hkv, 64, d).transpose(1, 2).reshape(B, Hkv, C * 64, d).contiguous()
                  for t in (kp, vp))
        ks = ksp.view(B, C, Hkv, d).transpose(1, 2).contiguous()
        sas.sas_decode_tree(q, kd, vd, kc, vc, i32(lens), ks, topk, **opt)
    qbar = q.double().view(B, Hkv, G, N, d).mean(2)
    klen = max(float(t.double().norm(dim=-1).max()) for t in (kp, kd))
    for b in range(B):
        n, c0 = ntok[b], lens[b] // 64  # five cached tokens past c0 blocks, at most 33 drafted
        own = table[b].long()
        s = scale * torch.einsum("rtd,crd->rtc", qbar[b], ksp[own[:c0]].double())
        want = s.argsort(dim=-1, descending=True, stable=True)[..., :topk].sort(-1)[0]
        assert torch.equal(idx[b, :, :n].long(), want[:, :n])
        assert (idx[b, :, n:] == -7).all() and (out[b, :, n:] == 3.0).all()
        if b % 7 != 0:
            continue
        logg = s.gather(2, want) - s.logsumexp(-1, keepdim=True)
        for i in (0, n // 2, n - 1):
            for r in range(Hkv):
                at, kept = own[want[r, i]], range(r * G, r * G + G)
                tail = own[c0]
                kk = torch.cat([kp[at, r].reshape(-1, d), kp[tail, r, :5], kd[b, r, :i + 1]]).double()
                vv = torch.cat([vp[at, r].reshape(-1, d), vp[tail, r, :5], vd[b, r, :i + 1]]).double()
                bias = torch.zeros(kk.shape[0], dtype=torch.float64, device=DEV)
                bias[:64 * topk] = logg[r, i].repeat_interleave(64)
                qq = q[b, list(kept), i].double()
                p = torch.softmax(scale * qq @ kk.T + bias, -1)
                o, mass = p @ vv, p @ vv.abs()
                dz = (d + 8) * U * scale * qq.norm(dim=-1, keepdim=True) * klen
                w = 2.0 ** -8 if dtype == "bf16" else 0.0
                tol = (4 * dz + (64 * (topk + 2) + 64) * U + w) * mass + HALF[dtype] * o.abs()
                # the gate's score: exact products, its softmax sum of c0 terms
                tol = tol + 2 * (c0 + 64) * U * mass
                assert ((out[b, list(kept), i].double() - o).abs() <= tol).all()
