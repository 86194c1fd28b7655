"""The serving calls on the GPU against the fp64 oracle, and together.

Tolerances, derived before the first run. u = 2^-24 is fp32's half step,
h = 2^-8 (bf16) or 2^-24 (fp32) the half step of a stored output.
  rotation  sine and cosine, amplitude included, are rounded once (u of their
            value; the phase's last bit, 2^-32 turns, is 1.5e-9); one product and
            the sum round once each. |dy| <= 3 u A (|x0| + |x1|) + 2^-29 A (...),
            below A (|x0| + |x1|) 2^-22.3; + h |y|.
  tree      a logit of d products is within dz = (d + 8) u scale |q| max |k|
            (plus the same for the score inside a gate); weights move by
            2 dz, their sum and the output's accumulation over n keys by
            (n + 64) u; bf16 caches round each weight once, 2^-8. With
            M = sum_j p_j |v_j| (the oracle's): |do| <= (4 dz + (n + 64) u + w) M
            + h |o|, w = 2^-8 for bf16 and 0 for fp32.
  summary   64 additions: 64 u mean|k| + h |mean|, of the keys as stored.
Indices, slots, tables and copied values are compared for equality.
"""
import numpy as np
import pytest
import torch

import serving_cases as S
from gated_block_sparse_b200 import rope, sas
from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(autouse=True)
def clean_status():
    sas.sas_device_status(clear=True)
    yield
    st, msg = sas.sas_device_status(clear=True)
    assert st == 0, msg


def np64(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


# ------------------------------------------------------------------ rotation
def rot_tol(x, y, rot, interleaved, amp, dtype):
    """Per element bound; passed-through elements are copied exactly."""
    a = np.zeros_like(y)
    half = rot // 2
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        a[..., i] = a[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    t = amp * a * 2.0 ** -22.3
    t[..., :rot] += HALF[dtype] * np.abs(y[..., :rot])
    return t


ROT = [  # dtype, B, Hq, Hkv, N, d, rot, interleaved, scaling, start
    ("bf16", 1, 4, 2, 1, 128, 128, False, "none", 0),
    ("bf16", 2, 6, 3, 65, 128, 64, True, "linear", 131071),
    ("bf16", 1, 1, 1, 257, 64, 64, False, "parts", 1048000),
    ("bf16", 2, 3, 1, 33, 64, 20, True, "base", 5),
    ("bf16", 1, 8, 1, 9, 128, 2, False, "none", 524287),
    ("f32", 2, 6, 2, 77, 64, 48, True, "linear", 0),
    ("f32", 1, 2, 2, 513, 128, 128, False, "parts", 1048000),
    ("f32", 3, 2, 0, 5, 128, 36, False, "none", 70000),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("c", ROT)
def test_rotary_matches_the_oracle(c, inverse):
    dtype, B, Hq, Hkv, N, d, rot, inter, scaling, start = c
    rng = np.random.Generator(np.random.PCG64(7 * N + rot))
    f, amp = rope.inv_freq(rot, scaling=scaling, factor=8.0 if scaling != "none" else 1.0)
    tq, q = S.rounded(rng.standard_normal((B, Hq, N, d)), dtype)
    tq, q = tq.reshape(B, Hq, N, d), q.reshape(B, Hq, N, d)
    tk = k = None
    if Hkv:
        tk, k = S.rounded(rng.standard_normal((B, Hkv, N, d)), dtype)
        tk, k = tk.reshape(B, Hkv, N, d).to(DEV), k.reshape(B, Hkv, N, d)
    st = np.array([start - 3 * b if start else 2 * b for b in range(B)])
    pos = st[:, None] + np.arange(N)
    amp32 = float(np.float32(amp))
    got = sas.sas_rotary(tq.to(DEV), f.to(DEV), k=tk, start=i32(st), interleaved=inter,
                         amplitude=amp, inverse=inverse)
    got = (got,) if k is None else got
    for g, x in zip(got, (q, k)):
        ref = SO.rotate(x, pos, f.double().numpy(), inter, amp32, inverse)
        err = np.abs(np64(g) - ref)
        assert (err <= rot_tol(x, ref, rot, inter, amp32, dtype)).all(), err.max()
    # given positions take the same path to the same bits
    again = sas.sas_rotary(tq.to(DEV), f.to(DEV), k=tk, pos=i32(pos), interleaved=inter,
                           amplitude=amp, inverse=inverse)
    again = (again,) if k is None else again
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype,rot", [("bf16", 128), ("bf16", 20), ("f32", 64)])
def test_rotary_reads_and_writes_strided_views(dtype, rot):
    B, N, Hq, Hkv, d = 2, 37, 4, 2, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).to(S.TORCH[dtype]).to(DEV)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    f = rope.inv_freq(rot)[0].to(DEV)
    want = sas.sas_rotary(q.contiguous(), f, k=k.contiguous())
    got = sas.sas_rotary(q, f, k=k)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # odd strides (no 16-byte rows) and a head shared by broadcasting
    wide = torch.randn((B, Hq, N, d + 3), generator=g).to(S.TORCH[dtype]).to(DEV)
    odd = wide[..., :d]
    shared = k[:, :1].expand(B, Hkv, N, d)
    a = sas.sas_rotary(odd, f, k=shared)
    b = sas.sas_rotary(odd.contiguous(), f, k=shared.contiguous())
    # the element-wise path rounds as the vector path does
    assert all(torch.equal(i, j) for i, j in zip(a, b))
    # into a view of a larger buffer, whose other rows stay, and in place
    buf = torch.full((B, N, Hq + 2 * Hkv, d), 9.0, dtype=q.dtype, device=DEV)
    out = (buf[:, :, :Hq].transpose(1, 2), buf[:, :, Hq:Hq + Hkv].transpose(1, 2))
    sas.sas_rotary(q, f, k=k, out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert (buf[:, :, Hq + Hkv:] == 9.0).all()
    y = x.clone()
    yq, yk = y[:, :, :Hq].transpose(1, 2), y[:, :, Hq:Hq + Hkv].transpose(1, 2)
    sas.sas_rotary(yq, f, k=yk, out=(yq, yk))
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])
    assert torch.equal(y[:, :, Hq + Hkv:], x[:, :, Hq + Hkv:])


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_backward_is_the_gradient(inter):
    """L = sum(dy . R x): the inverse call on dy against differences of L along
    single inputs (L is linear in x, so a difference of any width is exact up
    to rounding: 2 (2^-22.3 + u) A (|dy0| + |dy1|) per unit step)."""
    B, H, N, d, rot = 1, 2, 5, 64, 48
    f, amp = rope.inv_freq(rot, scaling="parts", factor=4.0)
    f = f.to(DEV)
    g = torch.Generator().manual_seed(11)
    x = torch.randn((B, H, N, d), generator=g).to(DEV)
    dy = torch.randn((B, H, N, d), generator=g).to(DEV)
    start = i32([90000])
    dx = sas.sas_rotary(dy, f, start=start, interleaved=inter, amplitude=amp, inverse=True)
    y0 = sas.sas_rotary(x, f, start=start, interleaved=inter, amplitude=amp)
    for e in (0, 1, 23, 24, 47, 48, 63):
        x1 = x.clone()
        x1[0, 1, 3, e] += 1.0
        y1 = sas.sas_rotary(x1, f, start=start, interleaved=inter, amplitude=amp)
        diff = float(((y1.double() - y0.double()) * dy.double()).sum())
        scale = amp * float(x[0, 1, 3].abs().max() + 1.0) * 2 * float(dy[0, 1, 3].abs().max())
        assert abs(diff - float(dx[0, 1, 3, e])) <= 8 * scale * 2.0 ** -22.3


def test_rotary_tree_positions_and_bad_parents():
    f = rope.inv_freq(128)[0].to(DEV)
    rng = np.random.Generator(np.random.PCG64(2))
    par = S.parents_of("tree", 3, 64, rng)
    q = torch.randn((3, 2, 64, 128), generator=torch.Generator().manual_seed(5)).to(DEV)
    start = np.array([0, 17, 500000])
    got = sas.sas_rotary(q, f, start=i32(start), parents=i32(par))
    want = sas.sas_rotary(q, f, pos=i32(start[:, None] + SO.depths(par)))
    assert torch.equal(got, want)
    par[1, 5], par[2, 0] = 9, -7  # a parent above its child, and nonsense: read as roots
    got = sas.sas_rotary(q, f, start=i32(start), parents=i32(par))
    st, msg = sas.sas_device_status(clear=True)
    assert st == 5 and "k_rotary" in msg
    par[1, 5], par[2, 0] = -1, -1
    assert torch.equal(got, sas.sas_rotary(q, f, pos=i32(start[:, None] + SO.depths(par))))


@pytest.mark.parametrize("rot", [64, 20])  # vectors and single elements
def test_rotary_near_quarter_turns(rot):
    """Angles at odd quarter turns, where the cosine is as small as the rounding of
    the fp32 frequency leaves it (1e-8 to 1e-3): x = (1, 0) turns to (cos, sin).
    Bound: 2^-52 of the angle, and one rounding of the cosine and of its product
    with 1 (2 u of it). The frequency in turns is a 64-bit fraction whose last bit
    is cut, so p positions add up to p 2^-64 turns, 2 pi p 2^-64 radians: a term
    of its own, since a small frequency's 2^-52 is less than that bit."""
    d, pos = 64, np.array([1, 3, 5, 4097, 65535, 1048575], dtype=np.int64)
    f = np.full(rot // 2, 0.3, dtype=np.float32)
    for i, p in enumerate(pos):
        f[i] = np.float32(np.pi / 2 / p)
    x = np.zeros((1, 1, len(pos), d))
    x[..., :rot // 2] = 1.0
    y = np64(sas.sas_rotary(torch.from_numpy(x).float().to(DEV), torch.from_numpy(f).to(DEV),
                            pos=i32(pos[None])))[0, 0]
    for i, p in enumerate(pos):
        theta = np.longdouble(f[i]) * np.longdouble(p)
        want = float(np.cos(theta))
        assert 0 < abs(want) < 1e-3
        tol = 2 * U * abs(want) + float(theta) * 2.0 ** -52 + 2 * np.pi * p * 2.0 ** -64
        assert abs(y[i, i] - want) <= tol, (p, y[i, i], want)


@pytest.mark.parametrize("dtype,rot", [("bf16", 64), ("f32", 64), ("bf16", 12)])
def test_rotary_of_frequencies_that_are_not_finite(dtype, rot):
    """An infinite or NaN frequency has no angle: its pair is NaN, in the rotation
    and in the cache write, and the other pairs are as before."""
    d, N = 64, 70
    g = torch.Generator().manual_seed(rot)
    x = torch.randn((1, 2, N, d), generator=g).to(S.TORCH[dtype]).to(DEV)
    f = rope.inv_freq(rot)[0]
    want = sas.sas_rotary(x, f.to(DEV))
    gone = torch.zeros(d, dtype=torch.bool)
    for p, v in ((0, float("nan")), (3, float("inf")), (rot // 2 - 1, float("-inf"))):
        f[p] = v
        gone[p] = gone[p + rot // 2] = True
    got = sas.sas_rotary(x, f.to(DEV)).cpu()
    kc, vc = (torch.zeros((1, 2, 128, d), dtype=x.dtype, device=DEV) for _ in range(2))
    sas.sas_cache_append(x, x, i32([0]), kc, vc, inv_freq=f.to(DEV))
    for y in (got, kc[:, :, :N].cpu()):
        assert torch.isnan(y[..., gone]).all()
        assert torch.equal(y[..., ~gone], want.cpu()[..., ~gone])
    assert torch.equal(vc[:, :, :N], x)


@pytest.mark.parametrize("N", [65, 1024])
def test_rotary_of_long_trees(N):
    """The longest tree that is taken: a chain, and a random tree beside it."""
    f = rope.inv_freq(64)[0].to(DEV)
    par = np.stack([np.arange(N) - 1, S.parents_of("tree", 1, N, np.random.Generator(
        np.random.PCG64(N)))[0]]).astype(np.int32)
    q = torch.randn((2, 3, N, 64), generator=torch.Generator().manual_seed(N)).to(DEV)
    got = sas.sas_rotary(q, f, start=i32([5, 900]), parents=i32(par))
    want = sas.sas_rotary(q, f, pos=i32(np.array([[5], [900]]) + SO.depths(par)))
    assert torch.equal(got, want)
    with pytest.raises(sas.SasError, match="1024 with parents"):
        sas.sas_rotary(q[:, :, :1].expand(2, 3, 1025, 64), f, parents=i32(np.full((2, 1025), -1)))


@pytest.mark.parametrize("N,Hkv", [(1, 2), (5, 1), (70, 2)])
def test_rotary_within_one_buffer(N, Hkv):
    """Inputs and outputs that alternate in one buffer without sharing a row are
    taken; a view shifted by a head or a token is refused."""
    B, Hq, d = 2, 4, 64
    g = torch.Generator().manual_seed(N)
    f, H = rope.inv_freq(d)[0].to(DEV), Hq + Hkv
    x = torch.randn((B, N, 2, H + 1, d), generator=g).bfloat16().to(DEV)
    keep = x.clone()
    heads = lambda t, lo, n: t[:, :, :, lo:lo + n].permute(2, 0, 3, 1, 4)  # [2][B][H][N][d]
    (q, qo), (k, ko) = heads(x, 0, Hq), heads(x, Hq, Hkv)
    want = sas.sas_rotary(q.contiguous(), f, k=k.contiguous())
    sas.sas_rotary(q, f, k=k, out=(qo, ko))
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert torch.equal(x[:, :, 0], keep[:, :, 0]) and torch.equal(x[:, :, 1, H], keep[:, :, 1, H])
    with pytest.raises(sas.SasError, match="an output must be"):
        sas.sas_rotary(q, f, k=k, out=(heads(x, 1, Hq)[0], ko))
    with pytest.raises(sas.SasError, match="qo and ko"):
        sas.sas_rotary(q, f, k=k, out=(qo, heads(x, Hq - 1, Hkv)[1]))
    if N > 2:
        with pytest.raises(sas.SasError, match="an output must be"):
            sas.sas_rotary(q[:, :, 1:], f, out=q[:, :, :-1])
    sas.sas_rotary(q, f, k=k, out=(q, k))  # in place
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, :, 0, H], keep[:, :, 0, H])


# ---------------------------------------------------------------- page tables
def page_case(seed, B, T, top, width=None, short=0):
    rng = np.random.Generator(np.random.PCG64(seed))
    lens = rng.integers(0, top + 1, B)
    nnew = rng.integers(0, T + 1, B)
    have, need = -(-lens // 64), -(-(lens + nnew) // 64) - (-(-lens // 64))
    width = width or int((top + T) // 64 + 2)
    npages = int(have.sum() + need.sum()) + 5
    perm = rng.permutation(npages).astype(np.int32)
    table = np.full((B, width), -5, dtype=np.int32)
    at = 0
    for b in range(B):
        n = min(int(have[b]), width)
        table[b, :n] = perm[at:at + n]
        at += n
    free = perm[at:at + int(need.sum()) + 2 - short]
    return lens.astype(np.int32), nnew.astype(np.int32), table, free, npages


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,T,top,short,head", [
    (1, 1, 0, 0, 0), (3, 1, 64, 0, 0), (1030, 1, 5000, 0, 0), (7, 16, 130, 3, 0),
    (5, 17, 200, 0, 0), (64, 100, 4096, 9, 2), (9, 1025, 300, 4, 1), (2, 4096, 63, 0, 0),
    (1, 64, 64, 0, 0)])
def test_page_map_matches_the_oracle(B, T, top, short, head, inplace):
    lens, nnew, table, free, npages = page_case(B * T + top, B, T, top, short=short)
    want = SO.page_map(lens, nnew, table, free, head, T, npages)
    tl, th, tt = i32(lens), i32([head]), i32(table)
    out = None
    if inplace:
        out = (torch.empty((B, T), dtype=torch.int32, device=DEV), tl,
               torch.empty(B, dtype=torch.int32, device=DEV), th)
    got = sas.sas_page_map(tl, i32(nnew), tt, i32(free), th, T, npages, out=out)
    for name, g, x in zip(("slots", "new_lens", "taken", "head", "table"), (*got, tt), want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(x)), x), name


@pytest.mark.parametrize("T", [8, 40])
def test_page_map_refuses_impossible_sequences(T):
    lens = np.array([10, -1, 60, 64 * 3, 0, 5], dtype=np.int32)
    nnew = np.array([T, 1, T + 1, 1, 2, -3], dtype=np.int32)
    table = np.arange(18, dtype=np.int32).reshape(6, 3)
    free = np.array([30, 31, 32], dtype=np.int32)
    want = SO.page_map(lens, nnew, table, free, 0, T, 40)
    tt = i32(table)
    got = sas.sas_page_map(i32(lens), i32(nnew), tt, i32(free), i32([0]), T, 40)
    for g, x in zip((*got, tt), want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(x)), x)
    assert got[2].tolist()[1:] == [-1, -1, -1, 1, -1]
    # ids outside the pool: written as listed, no slots, reported
    tt = i32(table)
    got = sas.sas_page_map(i32([70, 0]), i32([3, 2]), tt[:2].contiguous(), i32([99, 98]), i32([0]),
                           T, 1)
    st, msg = sas.sas_device_status(clear=True)
    assert st == 5 and "k_page" in msg
    assert (got[0] == -1).all() and got[1].tolist() == [73, 2]
    # an empty batch, and a head past its list
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    got = sas.sas_page_map(e, e, i32(np.zeros((0, 3))), i32([1]), i32([0]), T, 4)
    assert got[3].tolist() == [0]
    got = sas.sas_page_map(i32([0]), i32([1]), tt[:1].contiguous(), i32([1]), i32([5]), T, 40)
    assert got[2].tolist() == [-1] and got[3].tolist() == [5]
    assert sas.sas_device_status(clear=True)[0] == 5


# ---------------------------------------------------------------- cache write
APPEND = [  # dtype, sums, B, Hq, Hkv, T, d, lens, ntok, paged, rot, interleaved, rows, q
    ("bf16", "f32", 2, 8, 2, 1, 128, [63, 64], [1, 1], True, 128, False, False, True),
    ("bf16", "bf16", 3, 4, 1, 130, 128, [0, 1, 190], [130, 64, 0], True, 64, True, False, True),
    ("bf16", "f32", 1, 6, 2, 77, 64, [50], [77], False, 64, False, False, True),
    ("bf16", "bf16", 2, 3, 3, 20, 128, [60, 128], [9, 20], False, 0, False, True, False),
    ("f32", "f32", 2, 2, 2, 65, 64, [64, 5], [65, 60], False, 20, True, False, True),
    ("f32", "bf16", 1, 4, 4, 200, 128, [0], [200], True, 128, False, False, False),
    ("f32", "f32", 2, 2, 1, 64, 128, [127, 0], [1, 64], True, 36, False, True, False),
]


def append_case(c, seed=1):
    dtype, sums, B, Hq, Hkv, T, d, lens, ntok, paged, rot, inter, use_rows, use_q = c
    rng = np.random.Generator(np.random.PCG64(seed))
    C = (max(lens) + T) // 64 + 1
    shape = (B * C + 2, Hkv, 64, d) if paged else (B, Hkv, 64 * C, d)
    sshape = (B * C + 2, Hkv, d) if paged else (B, Hkv, C, d)
    x = {}
    for n, sh, dt in (("k", (B, Hkv, T, d), dtype), ("v", (B, Hkv, T, d), dtype),
                      ("q", (B, Hq, T, d), dtype), ("kc", shape, dtype), ("vc", shape, dtype),
                      ("ks", sshape, sums)):
        t, a = S.rounded(rng.standard_normal(sh), dt)
        x[n], x[n + "64"] = t.reshape(sh).to(DEV), a.reshape(sh)
    rows = None
    if use_rows:
        rows = rng.integers(0, T, (B, T)).astype(np.int32)
    slots = None
    if paged:
        pages = rng.permutation(B * C + 2)[:B * C].reshape(B, C)
        slots = np.full((B, T), -1, dtype=np.int32)
        for b in range(B):
            for j in range(ntok[b]):
                p = lens[b] + j
                slots[b, j] = pages[b, p // 64] * 64 + p % 64
        x["pages"] = pages
    x.update(rows=rows, slots=slots, f=rope.inv_freq(rot)[0] if rot else None)
    return x


@pytest.mark.parametrize("c", APPEND)
def test_cache_append_matches_the_oracle(c):
    dtype, sums, B, Hq, Hkv, T, d, lens, ntok, paged, rot, inter, use_rows, use_q = c
    x = append_case(c)
    f = x["f"]
    amp = 1.25 if rot else 1.0
    qo = torch.full((B, Hq, T, d), 7.0, dtype=x["q"].dtype, device=DEV) if use_q else None
    opt = dict(ksum=x["ks"], ntok=i32(ntok), rows=None if x["rows"] is None else i32(x["rows"]),
               slots=None if x["slots"] is None else i32(x["slots"]),
               inv_freq=None if f is None else f.to(DEV), interleaved=inter, amplitude=amp)
    sas.sas_cache_append(x["k"], x["v"], i32(lens), x["kc"], x["vc"],
                         q=x["q"] if use_q else None, out=qo, **opt)
    f64 = None if f is None else f.double().numpy()
    turn = None if f is None else (lambda y, p: SO.rotate(y, p, f64, inter, amp))
    kc, vc, _ = SO.append(x["k64"], x["v64"], lens, x["kc64"], x["vc64"], x["ks64"], ntok,
                          x["rows"], x["slots"], turn, lambda y: y, lambda y: y)
    assert np.array_equal(np64(x["vc"]), vc)
    got = np64(x["kc"])
    same = kc == x["kc64"]
    assert np.array_equal(got[same], kc[same])  # rows that no token names, and rot = 0
    if rot == 0:
        assert np.array_equal(got, kc)
    else:
        # a pair's two inputs are at most sqrt(2) of its rotated length
        big = np.abs(kc[..., :rot])
        pair = np.concatenate([big[..., rot // 2:], big[..., :rot // 2]], -1) if not inter else \
            big.reshape(*big.shape[:-1], -1, 2)[..., ::-1].reshape(big.shape)
        tol = 2 * (big + pair) * 2.0 ** -22.3 + HALF[dtype] * big
        assert (np.abs(got - kc)[..., :rot] <= tol).all()
        assert np.array_equal(got[..., rot:], kc[..., rot:])
    # summaries: the mean of the keys as they are now stored, where a block was completed
    ks = x["ks64"].copy()
    for b in range(B):
        for m in range(lens[b] // 64, (lens[b] + ntok[b]) // 64):
            keys = got[x["pages"][b, m]] if paged else got[b, :, 64 * m:64 * m + 64]
            at = x["pages"][b, m] if paged else (b, slice(None), m)
            ks[at] = keys.mean(1)
    tol = 64 * U * np.abs(got).max() + HALF[sums] * np.abs(ks)
    tol[ks == x["ks64"]] = 0.0
    assert (np.abs(np64(x["ks"]) - ks) <= tol).all()
    if use_q:
        pos = np.asarray(lens)[:, None] + np.arange(T)
        ref = SO.rotate(x["q64"], pos, f64, inter, amp)
        tol = rot_tol(x["q64"], ref, rot, inter, amp, dtype)
        assert (np.abs(np64(qo) - ref) <= tol).all()  # rows past ntok too


def test_cache_append_leaves_out_what_is_out_of_range():
    c = ("bf16", "f32", 3, 2, 2, 70, 64, [0, 64, 10], [70, 70, 70], True, 0, False, True, False)
    x = append_case(c)
    kc0, vc0, ks0 = x["kc"].clone(), x["vc"].clone(), x["ks"].clone()
    slots, rows = x["slots"].copy(), np.tile(np.arange(70, dtype=np.int32), (3, 1))
    slots[0, 5] = -1                      # left out quietly; its block keeps its summary
    slots[1, 3] = kc0.shape[0] * 64       # past the pool: reported
    rows[1, 64] = 70                      # past the rows: reported
    lens, ntok = [0, 64, 10], [70, 70, 71]  # and an impossible count: nothing of it
    sas.sas_cache_append(x["k"], x["v"], i32(lens), x["kc"], x["vc"], ksum=x["ks"],
                         ntok=i32(ntok), rows=i32(rows), slots=i32(slots))
    st, msg = sas.sas_device_status(clear=True)
    assert st == 5 and "k_append" in msg
    slots[1, 3] = slots[1, 64] = -1
    slots[2] = -1
    kc, vc, ks = SO.append(x["k64"], x["v64"], lens, np64(kc0), np64(vc0), np64(ks0),
                           [70, 70, 70], None, slots, None, lambda y: y, lambda y: y)
    assert np.array_equal(np64(x["kc"]), kc) and np.array_equal(np64(x["vc"]), vc)
    for b in range(2):  # both first blocks have a token left out
        assert torch.equal(x["ks"][x["pages"][b, b]], ks0[x["pages"][b, b]])
    # contiguous: tokens past the end of the cache
    c = ("f32", "f32", 1, 1, 1, 10, 64, [60], [10], False, 0, False, False, False)
    x = append_case(c)
    kc, vc, ks = (t[:, :, :64].contiguous() if t.dim() == 4 and t.shape[2] > 60 else t[:, :, :1].contiguous()
                  for t in (x["kc"], x["vc"], x["ks"]))
    sas.sas_cache_append(x["k"], x["v"], i32([60]), kc, vc, ksum=ks)
    assert sas.sas_device_status(clear=True)[0] == 5
    assert torch.equal(kc[:, :, 60:], x["k"][:, :, :4])
    assert torch.equal(vc[:, :, 60:], x["v"][:, :, :4])


@pytest.mark.parametrize("slot,reported", [(-1, False), (-2, True), (-64, True), (-2 ** 31, True)])
def test_cache_append_reports_slots_below_minus_one(slot, reported):
    c = ("bf16", "f32", 1, 2, 2, 70, 64, [0], [70], True, 0, False, False, False)
    x = append_case(c)
    kc0 = x["kc"].clone()
    slots = x["slots"].copy()
    slots[0, 5] = slot
    sas.sas_cache_append(x["k"], x["v"], i32([0]), x["kc"], x["vc"], ksum=x["ks"], slots=i32(slots))
    st, msg = sas.sas_device_status(clear=True)
    assert (st == 5 and "k_append" in msg) if reported else st == 0
    slots[0, 5] = -1
    kc, vc, _ = SO.append(x["k64"], x["v64"], [0], np64(kc0), x["vc64"], x["ks64"], [70], None,
                          slots, None, lambda y: y, lambda y: y)
    assert np.array_equal(np64(x["kc"]), kc) and np.array_equal(np64(x["vc"]), vc)


def test_cache_append_reports_positions_past_31_bits():
    """A length whose tokens would pass the largest int32 position, in a paged
    cache that does not look at it otherwise: left out; one token less is taken."""
    c = ("bf16", "f32", 1, 2, 2, 70, 64, [0], [70], True, 64, False, False, False)
    x = append_case(c)
    kc0, f = x["kc"].clone(), x["f"].to(DEV)
    args = (x["kc"], x["vc"])
    sas.sas_cache_append(x["k"], x["v"], i32([2 ** 31 - 70]), *args, slots=i32(x["slots"]), inv_freq=f)
    assert sas.sas_device_status(clear=True)[0] == 5 and torch.equal(x["kc"], kc0)
    sas.sas_cache_append(x["k"], x["v"], i32([2 ** 31 - 71]), *args, slots=i32(x["slots"]), inv_freq=f)
    assert sas.sas_device_status(clear=True)[0] == 0 and not torch.equal(x["kc"], kc0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_append_rotates_q_in_place_and_beside_the_cache(dtype):
    """qo = q, contiguous; k and v views of a projection that ends where the cache
    begins; and the refusal of k and v that lie in the cache."""
    B, Hq, Hkv, T, d, N = 2, 4, 2, 70, 64, 256
    dt = S.TORCH[dtype]
    g = torch.Generator().manual_seed(8)
    n = B * T * 2 * Hkv * d
    buf = torch.randn(n + 2 * B * Hkv * N * d, generator=g).to(dt).to(DEV)
    kv = buf[:n].view(B, T, 2 * Hkv, d)
    k, v = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
    kc, vc = buf[n:].view(2, B, Hkv, N, d)
    q = torch.randn((B, Hq, T, d), generator=g).to(dt).to(DEV)
    f, lens = rope.inv_freq(d)[0].to(DEV), i32([3, 100])
    kc2, vc2 = kc.clone(), vc.clone()
    want = sas.sas_cache_append(k.contiguous(), v.contiguous(), lens, kc2, vc2, inv_freq=f, q=q)
    assert sas.sas_cache_append(k, v, lens, kc, vc, inv_freq=f, q=q, out=q) is q
    assert torch.equal(q, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    for bad in (dict(k=kc[:, :, :T]), dict(v=kc[:, :, N - T:]), dict(k=vc[:, :, 9:9 + T])):
        with pytest.raises(sas.SasError, match="must not lie in the cache"):
            sas.sas_cache_append(**{**dict(k=k, v=v), **bad}, lens=lens, kc=kc, vc=vc)
    with pytest.raises(sas.SasError, match="kc and vc must not overlap"):
        sas.sas_cache_append(k, v, lens, kc, kc)


# ----------------------------------------------------------------------- tree
TREE = [  # dtype, sums, B, Hq, Hkv, d, T, N, lens, ntok, topk, gated, kind, paged
    ("f32", "f32", 2, 2, 2, 64, 7, 640, [600, 321], None, 2, 1, "tree", False),
    ("f32", "f32", 3, 6, 2, 64, 64, 512, [0, 1, 447], [64, 3, 64], 3, 0, "chain", False),
    ("f32", "bf16", 2, 8, 1, 128, 13, 1024, [1024, 130], [13, 5], 31, 1, "tree", True),
    ("f32", "f32", 1, 3, 3, 128, 64, 576, [575], None, 4, 1, "chain", True),
    ("f32", "f32", 1, 4, 1, 64, 5, 256, [200], None, 0, 1, "tree", False),
    ("bf16", "f32", 1, 8, 2, 128, 4, 4096, [4000], None, 15, 1, "chain", False),
    ("bf16", "f32", 3, 4, 1, 128, 64, 1024, [63, 64, 1000], [64, 0, 33], 5, 1, "chain", False),
    ("bf16", "bf16", 2, 8, 1, 128, 64, 2112, [2100, 2111], None, 7, 1, "tree", True),
    ("bf16", "f32", 2, 6, 2, 64, 19, 1024, [1023, 0], None, 3, 0, "tree", True),
    ("bf16", "bf16", 1, 5, 1, 64, 33, 704, [690], None, 128, 1, "flat", False),
    ("bf16", "f32", 1, 2, 2, 128, 1, 640, [640], None, 3, 1, "chain", False),
    ("bf16", "f32", 2, 2, 1, 64, 64, 128, [1, 127], None, 0, 1, "chain", True),
    ("bf16", "f32", 1, 7, 1, 128, 50, 8192, [8100], None, 40, 1, "tree", False),
    # short caches: one, two and four copies of the rows
    ("bf16", "bf16", 2, 8, 1, 128, 33, 128, [127, 40], [33, 20], 2, 1, "tree", True),
    ("bf16", "f32", 3, 4, 1, 64, 13, 128, [64, 128, 0], [13, 2, 7], 5, 1, "chain", False),
    ("bf16", "f32", 1, 2, 2, 128, 9, 512, [480], None, 0, 1, "tree", False),
    ("f32", "f32", 2, 6, 2, 128, 9, 128, [100, 1], None, 1, 1, "tree", False),
]


def tree_call(x, topk, gated, paged, out=None, idx=None, **kw):
    kc, vc, ks, table = x["kc_t"], x["vc_t"], x["ksum_t"], None
    if paged:
        kc, vc, ks, table = S.to_pages(x, x["rng"])
        table = table.to(DEV)
    return sas.sas_decode_tree(
        x["q_t"].to(DEV), x["kd_t"].to(DEV), x["vd_t"].to(DEV), kc.to(DEV), vc.to(DEV),
        i32(x["lens"]), ks.to(DEV), topk, parents=i32(x["parents"]), ntok=i32(x["ntok"]),
        block_table=table, gated=gated, out=out, idx_out=idx, **kw)


def tree_tol(x, o, mass, topk, dtype, sums):
    d, B = x["q"].shape[-1], x["q"].shape[0]
    scale = 1.0 / np.sqrt(d)
    # sum_c |q_c k_c| <= |q| |k|; the largest key stands for all
    finite = [np.where(np.isfinite(x[n]), x[n], 0.0) for n in ("kc", "kd")]
    klen = max(np.sqrt((k * k).sum(-1)).max() for k in finite)
    kmax = max(np.abs(k).max() for k in finite)
    dz = (d + 8) * U * scale * np.sqrt((x["q"] ** 2).sum(-1, keepdims=True)) * klen
    if sums == "bf16":
        # the fp32 and the fp64 mean of a block filled by a path may round to
        # neighbouring bf16 values in one element: a score off by one step there
        dz = dz + scale * np.abs(x["q"]).max() * kmax * 2.0 ** -8 * (2.0 ** -3)
    n = 64 * (topk + 2)
    w = 2.0 ** -8 if dtype == "bf16" else 0.0
    return (4 * dz + (n + 64) * U + w) * mass + HALF[dtype] * np.abs(o)


def check_tree(x, got, idx, topk, gated, dtype, sums):
    o, want_idx, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"],
                                       x["ksum"], x["parents"], x["ntok"], topk, gated,
                                       S.store(sums))
    B, _, T, _ = o.shape
    got, idx = np64(got), idx.cpu().numpy()
    for b in range(B):
        n = int(x["ntok"][b])
        assert np.array_equal(idx[b, :, :n], want_idx[b, :, :n])
        err = np.abs(got[b, :, :n] - o[b, :, :n])
        tol = tree_tol(x, np.nan_to_num(o), np.nan_to_num(mass), topk, dtype, sums)[b, :, :n]
        assert (err <= tol).all(), (float(err.max()), float((err - tol).max()))
        # rows behind the last token are left as they were
        assert (got[b, :, n:] == 3.0).all() and (idx[b, :, n:] == -7).all()


@pytest.mark.parametrize("c", TREE)
def test_decode_tree_matches_stepwise_decode(c):
    dtype, sums, B, Hq, Hkv, d, T, N, lens, ntok, topk, gated, kind, paged = c
    x = S.tree_case(100 + T + N, B, Hq, Hkv, d, T, N, lens, topk, dtype, sums, kind, ntok)
    out = torch.full((B, Hq, T, d), 3.0, dtype=S.TORCH[dtype], device=DEV)
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    tree_call(x, topk, gated, paged, out, idx)
    check_tree(x, out, idx, topk, gated, dtype, sums)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_tree_ignores_what_a_token_does_not_see(dtype, paged):
    """NaN and infinities in cached rows behind the end, in drafted rows behind
    the last, in siblings, and in a block that only some tokens keep."""
    B, Hq, Hkv, d, T, N, topk = 2, 4, 2, 128, 12, 1024, 4
    x = S.tree_case(9, B, Hq, Hkv, d, T, N, [900, 963], topk, dtype, "f32", "tree", [12, 9])
    clean = S.tree_case(9, B, Hq, Hkv, d, T, N, [900, 963], topk, dtype, "f32", "tree", [12, 9])
    _, sel, _ = SO.decode_tree(clean["q"], clean["kd"], clean["vd"], clean["kc"], clean["vc"],
                               clean["lens"], clean["ksum"], clean["parents"], clean["ntok"], topk)
    bad = [float("nan"), float("inf"), float("-inf")]
    hit = 0
    for b in range(B):
        n = int(x["lens"][b])
        for name in ("kc", "vc"):
            x[name][b, :, n:] = np.nan
            x[name + "_t"][b, :, n:] = bad[b]
        m = int(x["ntok"][b])
        for name in ("kd", "vd"):
            x[name][b, :, m:] = np.nan
            x[name + "_t"][b, :, m:] = bad[b]
        leaf = m - 1  # the last token: an ancestor of no other
        x["kd"][b, :, leaf] = x["vd"][b, :, leaf] = np.inf
        x["kd_t"][b, :, leaf] = x["vd_t"][b, :, leaf] = float("inf")
        # a value of a block that only some tokens keep
        blocks = [set(sel[b, 0, i][sel[b, 0, i] >= 0].tolist()) for i in range(m - 1)]
        some = sorted(set.union(*blocks) - set.intersection(*blocks))
        some = [s for s in some if s < n // 64]
        if some:
            hit += 1
            x["vc"][b, 0, 64 * some[0] + 5, 7] = np.inf
            x["vc_t"][b, 0, 64 * some[0] + 5, 7] = float("inf")
    assert hit
    out = torch.full((B, Hq, T, d), 3.0, dtype=S.TORCH[dtype], device=DEV)
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    tree_call(x, topk, 1, paged, out, idx)
    with np.errstate(invalid="ignore"):
        o, want_idx, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"],
                                           x["ksum"], x["parents"], x["ntok"], topk)
    got = np64(out)
    tol = tree_tol(x, np.nan_to_num(o), np.nan_to_num(mass, posinf=0.0), topk, dtype, "f32")
    for b in range(B):
        m = int(x["ntok"][b]) - 1
        fin = np.isfinite(o[b, :, :m])
        assert fin.any() and np.array_equal(np.isfinite(got[b, :, :m]), fin)
        assert (np.abs(got[b, :, :m][fin] - o[b, :, :m][fin]) <= tol[b, :, :m][fin]).all()
        assert np.array_equal(idx.cpu().numpy()[b, :, :m], want_idx[b, :, :m])
        assert (got[b, :, m + 1:] == 3.0).all()


@pytest.mark.parametrize("Hq,d,T", [(8, 64, 40), (8, 128, 7), (4, 128, 13)])
def test_decode_tree_keeps_the_weights_of_bf16_caches(Hq, d, T):
    """A weight goes to its product in two bf16 parts: the upper half of its
    bits, then the rest, below 2^-7 of it, rounded by half a step, so
    w = 2^-16 in the bound above. Few keys and short queries keep the other
    terms small: one part would pass the bound by several times."""
    x = S.tree_case(500 + T, 3, Hq, 1, d, T, 128, [0, 3, 66], 1, "bf16", "f32", "tree")
    x["q"] *= 0.125
    x["q_t"] *= 0.125
    got = np64(tree_call(x, 1, 1, False))
    o, _, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"], x["ksum"],
                                x["parents"], x["ntok"], 1)
    tol = tree_tol(x, o, mass, 1, "bf16", "f32") + (2.0 ** -16 - 2.0 ** -8) * mass
    assert (np.abs(got - o) <= tol).all()


@pytest.mark.parametrize("topk", [4, 40])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), 3.4e38])
@pytest.mark.parametrize("dtype,sums,paged", [("bf16", "f32", False), ("bf16", "bf16", True),
                                              ("f32", "f32", True), ("f32", "bf16", False)])
def test_decode_tree_with_an_infinite_summary(dtype, sums, paged, bad, topk):
    """A summary with one element that is infinite, or finite but past the
    largest bf16 value, and queries of the other sign there: its score is -inf
    (or hugely negative), its weight 0, and every result is finite, as in a
    decode step. With queries of the same sign the gated rows of that head are
    NaN for an infinity, and the other heads' are not."""
    B, Hq, Hkv, d, T, N, e = 2, 4, 2, 128, 9, 1024, 5
    if bad == 3.4e38 and sums == "bf16":
        bad = 3.38e38  # the largest magnitude that stays finite in bf16
    x = S.tree_case(41, B, Hq, Hkv, d, T, N, [900, 963], topk, dtype, sums, "tree", [9, 7])
    # the other blocks have nothing there, so the planted levels keep their order
    x["ksum"][..., e] = 0.0
    x["ksum_t"][..., e] = 0.0
    away = -np.sign(bad) * (np.abs(x["q"][..., e]) + 0.25)
    t, v = S.rounded(away, dtype)
    x["q_t"][..., e], x["q"][..., e] = t.reshape(away.shape), v.reshape(away.shape)
    x["ksum_t"][0, 0, 3, e] = bad
    x["ksum"][0, 0, 3, e] = float(x["ksum_t"][0, 0, 3, e])
    out = torch.full((B, Hq, T, d), 3.0, dtype=S.TORCH[dtype], device=DEV)
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    tree_call(x, topk, 1, paged, out, idx)
    check_tree(x, out, idx, topk, 1, dtype, sums)
    if not np.isinf(bad):
        return
    x["q_t"][..., e], x["q"][..., e] = -x["q_t"][..., e], -x["q"][..., e]
    out.fill_(3.0)
    tree_call(x, topk, 1, paged, out, idx)
    assert torch.isnan(out[0, :2, :9]).all()
    assert torch.isfinite(out[0, 2:, :9]).all() and torch.isfinite(out[1, :, :7]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,topk", [(1024, 5), (700 * 64, 33), (1300 * 64, 128)])
def test_decode_tree_ties_go_to_the_lower_block(dtype, N, topk):
    """Equal summaries: every score ties and the first blocks are kept; with a
    better block in the middle, it and the first ones (few and many ties: the
    list of candidates and the threshold by bits)."""
    B, Hq, Hkv, d, T = 1, 2, 1, 64, 3
    q = torch.randn((B, Hq, T, d), generator=torch.Generator().manual_seed(1)).abs() + 0.1
    q = q.to(S.TORCH[dtype]).to(DEV)
    kd = torch.zeros((B, Hkv, T, d), dtype=q.dtype, device=DEV)
    kc = torch.zeros((B, Hkv, N, d), dtype=q.dtype, device=DEV)
    ks = torch.full((B, Hkv, N // 64, d), 0.25, device=DEV)
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    o = sas.sas_decode_tree(q, kd, kd, kc, kc, i32([N - 20]), ks, topk, idx_out=idx)
    assert (idx.cpu() == torch.arange(topk, dtype=torch.int32)).all() and (o == 0).all()
    mid = N // 64 - 2
    ks[:, :, mid] = 0.5
    sas.sas_decode_tree(q, kd, kd, kc, kc, i32([N - 20]), ks, topk, idx_out=idx)
    want = list(range(topk - 1)) + [mid]
    assert (idx.cpu() == torch.tensor(want, dtype=torch.int32)).all()


@pytest.mark.parametrize("spread", [1.0, 1e3, 1e6])
def test_decode_tree_selects_beside_far_outliers(spread):
    """A few blocks score far above the others (up to a million times their
    spread): the kept set is still that of a stable sort. Scores are exact
    here: one nonzero element a query and distinct summaries on a 2^-8 grid."""
    B, Hkv, d, T, C, topk = 1, 2, 64, 5, 6000, 40
    rng = np.random.Generator(np.random.PCG64(int(spread)))
    q = torch.zeros((B, Hkv, T, d))
    q[..., 3] = 1.0
    lev = np.stack([rng.permutation(C) for _ in range(Hkv)]).astype(np.float64) / 256.0
    for r in range(Hkv):
        lev[r, rng.choice(C, 3, replace=False)] += 32.0 * spread
    ks = torch.zeros((B, Hkv, C, d))
    ks[0, :, :, 3] = torch.from_numpy(lev).float()
    kd = torch.zeros((B, Hkv, T, d))
    kc = torch.zeros((B, Hkv, C * 64, d))
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    sas.sas_decode_tree(q.to(DEV), kd.to(DEV), kd.to(DEV), kc.to(DEV), kc.to(DEV), i32([C * 64 - 64]),
                        ks.to(DEV), topk, scale=1.0, idx_out=idx)
    lev32 = ks[0, :, :C - 1, 3].numpy()  # one block is not whole yet
    for r in range(Hkv):
        want = np.sort(np.argsort(-lev32[r], kind="stable")[:topk])
        assert (idx[0, r].cpu().numpy() == want).all()


def test_decode_tree_of_one_token_is_a_decode_step():
    """T = 1 against sas_decode on the cache with the token appended; the same
    definition on two kernels, each within the tree's bound of it."""
    B, Hq, Hkv, d, N, topk = 3, 8, 2, 128, 2048, 7
    x = S.tree_case(21, B, Hq, Hkv, d, 1, N, [2000, 64, 1], topk, "bf16", "f32", "chain")
    one = tree_call(x, topk, 1, False)
    kc, vc = x["kc_t"].to(DEV), x["vc_t"].to(DEV)
    ks = x["ksum_t"].to(DEV)
    lens = i32(x["lens"])
    sas.sas_cache_append(x["kd_t"].to(DEV), x["vd_t"].to(DEV), lens, kc, vc, ksum=ks)
    step = sas.sas_decode(x["q_t"][:, :, 0].contiguous().to(DEV), kc, vc, lens + 1, ks, topk)
    o, _, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"], x["ksum"],
                                x["parents"], x["ntok"], topk)
    tol = 2 * tree_tol(x, o, mass, topk, "bf16", "f32")[:, :, 0]
    assert (np.abs(np64(one)[:, :, 0] - np64(step)) <= tol).all()


def test_decode_tree_reports_bad_parents_pages_and_lengths():
    B, Hq, Hkv, d, T, N, topk = 1, 4, 1, 128, 8, 512, 3
    x = S.tree_case(6, B, Hq, Hkv, d, T, N, [400], topk, "bf16", "f32", "chain")
    par = x["parents"].copy()
    x["parents"][0, 4] = 6
    o = tree_call(x, topk, 1, False)
    st, msg = sas.sas_device_status(clear=True)
    assert st == 5 and "k_tree_select" in msg and torch.isfinite(o.float()).all()
    x["parents"] = par
    kp, vp, ksp, table = S.to_pages(x, x["rng"])
    kp, vp, ksp = (torch.nan_to_num(t) for t in (kp, vp, ksp))
    table[0, 1], table[0, 6] = 10 ** 6, -4  # a history block and the tail's
    o = sas.sas_decode_tree(x["q_t"].to(DEV), x["kd_t"].to(DEV), x["vd_t"].to(DEV), kp.to(DEV),
                            vp.to(DEV), i32([400]), ksp.to(DEV), topk, block_table=table.to(DEV))
    st, msg = sas.sas_device_status(clear=True)
    assert st == 5 and torch.isfinite(o.float()).all()
    for lens, ntok in (([513], [8]), ([-1], [8]), ([400], [9])):
        x["lens"], x["ntok"] = np.array(lens), np.array(ntok)
        tree_call(x, topk, 1, False)
        assert sas.sas_device_status(clear=True)[0] == 5
    for dtype in ("bf16", "f32"):  # without a selection too
        x = S.tree_case(6, B, Hq, Hkv, d, T, N, [513], 1, dtype, "f32", "chain")
        tree_call(x, 0, 1, False)
        assert sas.sas_device_status(clear=True)[0] == 5
        x["lens"], x["parents"] = np.array([400]), par + 2
        tree_call(x, 0, 1, False)
        assert sas.sas_device_status(clear=True)[0] == 5


def masked_by_summary(x, dtype, sums, e=5):
    """Column e of every query positive and of every summary 0, so that a summary
    of -inf there gives a score of -inf in the oracle."""
    x["ksum"][..., e] = 0.0
    x["ksum_t"][..., e] = 0.0
    t, v = S.rounded(np.abs(x["q"][..., e]) + 0.25, dtype)
    x["q_t"][..., e] = t.reshape(x["q_t"][..., e].shape)
    x["q"][..., e] = v.reshape(x["q"][..., e].shape)


@pytest.mark.parametrize("where", [[10 ** 6, -4], [-1, 14]])
@pytest.mark.parametrize("topk", [4, 40])
@pytest.mark.parametrize("dtype,sums", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"),
                                        ("f32", "bf16")])
def test_decode_tree_leaves_out_pages_outside_the_pool(dtype, sums, topk, where):
    """Blocks whose page ids lie outside the pool score -inf and are not attended
    to; no other page (page 0 holds NaN) is read in their place."""
    B, Hq, Hkv, d, T, N, e = 2, 4, 2, 64, 12, 512, 5
    x = S.tree_case(61, B, Hq, Hkv, d, T, N, [420, 447], topk, dtype, sums, "tree", [12, 9])
    masked_by_summary(x, dtype, sums)
    kp, vp, ksp, table = S.to_pages(x, x["rng"], spare=0)
    nan = lambda t: torch.cat([torch.full_like(t[:1], float("nan")), t]).to(DEV)[:17]
    kp, vp, ksp, table = nan(kp), nan(vp), nan(ksp), table + 1
    npages, gone = kp.shape[0], [(0, 1), (1, 2)]
    for (b, m), w in zip(gone, where):
        table[b, m] = w if w != 14 else npages
        x["ksum"][b, :, m, e] = -np.inf
    out = torch.full((B, Hq, T, d), 3.0, dtype=S.TORCH[dtype], device=DEV)
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    sas.sas_decode_tree(x["q_t"].to(DEV), x["kd_t"].to(DEV), x["vd_t"].to(DEV), kp, vp,
                        i32(x["lens"]), ksp, topk, parents=i32(x["parents"]), ntok=i32(x["ntok"]),
                        block_table=table.to(DEV), out=out, idx_out=idx)
    st, msg = sas.sas_device_status(clear=True)
    assert st == 5 and "k_tree_scores" in msg
    check_tree(x, out, idx, topk, 1, dtype, sums)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_tree_leaves_out_a_tail_page_outside_the_pool(dtype):
    """Without a selection a token then attends to its path alone, as on an
    empty cache; with one, a path that fills the tail's block does not keep it."""
    B, Hq, Hkv, d, T, N, topk, e = 1, 4, 2, 64, 9, 256, 3, 5
    x = S.tree_case(62, B, Hq, Hkv, d, T, N, [100], topk, dtype, "f32", "tree")
    masked_by_summary(x, dtype, "f32")
    kp, vp, ksp, table = S.to_pages(x, x["rng"], spare=0)
    nan = lambda t: torch.cat([torch.full_like(t[:1], float("nan")), t]).to(DEV)
    kp, vp, ksp, table = nan(kp), nan(vp), nan(ksp), table + 1
    out = torch.full((B, Hq, T, d), 3.0, dtype=S.TORCH[dtype], device=DEV)

    def call(lens, k, idx=None):
        sas.sas_decode_tree(x["q_t"].to(DEV), x["kd_t"].to(DEV), x["vd_t"].to(DEV), kp, vp,
                            i32(lens), ksp, k, parents=i32(x["parents"]),
                            block_table=table.to(DEV), out=out, idx_out=idx)
        assert sas.sas_device_status(clear=True)[0] == 5
    table[0, 1] = -9
    call([100], 0)
    check_tree(dict(x, lens=np.array([0])), out, torch.empty((B, Hkv, T, 0), dtype=torch.int32), 0, 1,
               dtype, "f32")
    # 127 cached tokens: every token but the roots has filled block 1, which
    # stands at -inf in the oracle through the summary that the path gives it
    deep = SO.depths(x["parents"])[0] > 0
    assert deep.any()
    x["lens"] = np.array([127])
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    call([127], topk, idx)

    def gone(mean):
        mean = mean.copy()
        mean[..., e] = -np.inf
        return mean
    o, want, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"], x["ksum"],
                                   x["parents"], x["ntok"], topk, 1, gone)
    tol = tree_tol(x, o, mass, topk, dtype, "f32")
    assert (np.abs(np64(out) - o) <= tol)[:, :, deep].all()
    assert np.array_equal(idx.cpu().numpy()[:, :, deep], want[:, :, deep])


@pytest.mark.parametrize("topk", [0, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,ntok", [(513, 8), (-1, 8), (400, 9), (400, -2)])
def test_decode_tree_leaves_out_impossible_lengths(lens, ntok, dtype, topk):
    B, Hq, Hkv, d, T, N = 2, 4, 1, 64, 8, 512
    x = S.tree_case(63, B, Hq, Hkv, d, T, N, [400, 300], max(topk, 1), dtype, "f32", "chain")
    x["lens"], x["ntok"] = np.array([lens, 300]), np.array([ntok, 7])
    out = torch.full((B, Hq, T, d), 3.0, dtype=S.TORCH[dtype], device=DEV)
    idx = torch.full((B, Hkv, T, topk), -7, dtype=torch.int32, device=DEV)
    tree_call(x, topk, 1, False, out, idx)
    assert sas.sas_device_status(clear=True)[0] == 5
    assert (out[0] == 3.0).all() and (idx[0] == -7).all()
    y = {n: (v[1:] if n != "rng" else v) for n, v in x.items()}
    check_tree(y, out[1:], idx[1:], topk, 1, dtype, "f32")


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,T", [(4, 5), (8, 7), (8, 17)])  # 20, 56 and 136 rows a group
def test_decode_tree_of_caches_with_bad_values(Hq, T, d, paged):
    """Infinities and NaN where tokens do see them: a value of a kept block and
    one of the tail reach their column alone, a NaN key makes the rows that keep
    its block NaN and no others, also across splits and copies of the rows."""
    B, Hkv, N, topk = 2, 1, 1024, 4
    x = S.tree_case(71, B, Hq, Hkv, d, T, N, [900, 963], topk, "bf16", "f32", "tree", [T, T - 1])
    _, sel, _ = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"], x["ksum"],
                               x["parents"], x["ntok"], topk)
    inf, nan = float("inf"), float("nan")
    for b in range(B):
        n = int(x["lens"][b])
        blocks = [set(sel[b, 0, i][sel[b, 0, i] >= 0].tolist()) for i in range(int(x["ntok"][b]))]
        some = sorted(s for s in set.union(*blocks) - set.intersection(*blocks) if s < n // 64)
        both = sorted(s for s in set.intersection(*blocks) if s < n // 64)
        assert some
        for name, at, c, v in [("kc", 64 * some[0] + 9, 3, nan), ("vc", 64 * some[-1] + 33, 11, inf),
                               ("vc", n - 2, 7, -inf), ("vd", T - 2, 20, inf)] + \
                [("vc", 64 * m + 63, 30, inf) for m in both[:1]]:
            x[name][b, 0, at, c] = v
            x[name + "_t"][b, 0, at, c] = v
    out = torch.full((B, Hq, T, d), 3.0, dtype=torch.bfloat16, device=DEV)
    tree_call(x, topk, 1, paged, out)
    with np.errstate(invalid="ignore"):
        o, _, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"],
                                    x["ksum"], x["parents"], x["ntok"], topk)
    got = np64(out)
    finite = dict(x, kc=np.nan_to_num(x["kc"]))
    tol = tree_tol(finite, np.nan_to_num(o, posinf=0, neginf=0),
                   np.nan_to_num(mass, posinf=0, neginf=0), topk, "bf16", "f32")
    for b in range(B):
        m = int(x["ntok"][b])
        g, r = got[b, :, :m], o[b, :, :m]
        fin = np.isfinite(r)
        assert fin.any() and np.isnan(r).any() and np.isinf(r).any()
        assert np.array_equal(np.isnan(g), np.isnan(r))
        assert np.array_equal(g[np.isinf(r)], r[np.isinf(r)])
        assert (np.abs(g[fin] - r[fin]) <= tol[b, :, :m][fin]).all()


def test_binding_refuses_other_types_shapes_and_layouts():
    q = torch.zeros(1, 2, 4, 64, device=DEV)
    f = torch.ones(16, device=DEV)
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError, match="unsupported dtype"):
        sas.sas_rotary(q.half(), f)
    with pytest.raises(TypeError, match="inv_freq"):
        sas.sas_rotary(q, f.double())
    with pytest.raises(ValueError, match="inv_freq is on cpu"):
        sas.sas_rotary(q, f.cpu())
    with pytest.raises(ValueError, match="pos must have shape"):
        sas.sas_rotary(q, f, pos=i)
    with pytest.raises(ValueError, match="rows of q must be contiguous"):
        sas.sas_rotary(q.transpose(2, 3), f)
    with pytest.raises(TypeError, match="start must be"):
        sas.sas_rotary(q, f, start=i.long())
    with pytest.raises(ValueError, match="ko must have shape"):
        sas.sas_rotary(q, f, k=q, out=(q, q[:, :1]))
    with pytest.raises(ValueError, match="block_table must be contiguous"):
        sas.sas_page_map(i, i, torch.zeros(1, 6, dtype=torch.int32, device=DEV)[:, ::2], i, i, 1, 1)
    with pytest.raises(ValueError, match="vc must have shape"):
        sas.sas_cache_append(q, q, i, torch.zeros(1, 2, 64, 64, device=DEV), q)
    with pytest.raises(ValueError, match="out goes with q"):
        sas.sas_cache_append(q, q, i, q, q, out=q)
    with pytest.raises(ValueError, match="kd must have shape"):
        sas.sas_decode_tree(q, q[:, :, :3], q, q, q, i, None, 0)


def test_outputs_of_a_call_are_ordinary_tensors():
    """Outputs carved from one allocation: contiguous, aligned, apart, usable by
    torch, and any of them may be supplied instead."""
    q, k = torch.randn(1, 3, 5, 64, device=DEV), torch.randn(1, 1, 5, 64, device=DEV)
    f = rope.inv_freq(64)[0].to(DEV)
    qo, ko = sas.sas_rotary(q, f, k=k)
    assert qo.is_contiguous() and ko.is_contiguous() and ko.data_ptr() % 16 == 0
    assert qo.shape == q.shape and ko.shape == k.shape
    mine = torch.empty_like(k)
    q2, k2 = sas.sas_rotary(q, f, k=k, out=(None, mine))
    assert k2 is mine and torch.equal(q2, qo) and torch.equal(k2, ko)
    keep = qo.clone()
    ko.zero_()
    assert torch.equal(qo, keep) and torch.equal(qo.transpose(1, 2).reshape(-1), keep.transpose(1, 2).reshape(-1))
    del qo
    torch.cuda.empty_cache()
    assert (ko + 1 == 1).all()
    lens = i32([3, 0, 70])
    new = torch.empty_like(lens)
    out = sas.sas_page_map(lens, i32([1, 0, 2]), i32(np.arange(6).reshape(3, 2)), i32([7, 8]), i32([0]),
                           3, 9, out=(None, new, None, None))
    assert out[1] is new and new.tolist() == [4, 0, 72]
    assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in out)
    assert [tuple(t.shape) for t in out] == [(3, 3), (3,), (3,), (1,)]
    assert out[0].tolist() == [[3, -1, -1], [-1] * 3, [5 * 64 + 6, 5 * 64 + 7, -1]]


def test_kept_outputs_do_not_hold_large_ones():
    """The head or the lengths of a page map, or one tensor of a rotation, kept
    after a large call: memory of the others is free again."""
    def held(make):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        keep = make()
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated() - before, keep
    B, T = 64, 8192
    z = i32(np.zeros(B))
    args = (z, z, i32(np.zeros((B, 1))), i32([0]), i32([0]), T, 8)
    for i, most in ((1, 4 * 4096), (2, 4 * 4096), (3, 4 * 4096), (0, 4 * B * T + 512)):
        n, keep = held(lambda: sas.sas_page_map(*args)[i])
        assert n <= most and keep.untyped_storage().nbytes() <= most
    n, keep = held(lambda: sas.sas_page_map(z[:4], z[:4], i32(np.zeros((4, 1))), *args[3:5], 9, 8)[3])
    assert n <= 4 * 4096
    f = rope.inv_freq(128)[0].to(DEV)
    x = torch.zeros((1, 10, 4096, 128), dtype=torch.bfloat16, device=DEV)
    for i, H in ((0, 8), (1, 2)):
        n, keep = held(lambda: sas.sas_rotary(x[:, :8], f, k=x[:, 8:])[i])
        assert n <= H * 4096 * 256 + 512 and keep.untyped_storage().nbytes() == H * 4096 * 256


# ------------------------------------------------------------ streams, graphs
def test_calls_on_another_stream_and_in_graphs():
    B, Hq, Hkv, d, T, N, topk = 2, 4, 2, 128, 6, 1024, 4
    x = S.tree_case(31, B, Hq, Hkv, d, T, N, [700, 512], topk, "bf16", "f32", "tree")
    t = {n: x[n + "_t"].to(DEV) for n in ("q", "kd", "vd", "kc", "vc", "ksum")}
    lens, par = i32(x["lens"]), i32(x["parents"])
    f = rope.inv_freq(d)[0].to(DEV)

    def step():
        q, k = sas.sas_rotary(t["q"], f, k=t["kd"], start=lens, parents=par)
        o = sas.sas_decode_tree(q, k, t["vd"], t["kc"], t["vc"], lens, t["ksum"], topk, parents=par)
        kc, vc, ks = t["kc"].clone(), t["vc"].clone(), t["ksum"].clone()
        sas.sas_cache_append(k, t["vd"], lens, kc, vc, ksum=ks)
        return o, kc, vc, ks
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = sas.sas_decode_tree(*(sas.sas_rotary(t["q"], f, k=t["kd"], start=lens, parents=par,
                                             stream=side)), t["vd"], t["kc"], t["vc"], lens,
                            t["ksum"], topk, parents=par, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0])
    graphs, outs = [], []
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step())
        graphs.append(g)
    # new numbers in the same buffers, replayed in turn
    t["q"].copy_(t["q"].flip(2))
    lens.copy_(i32([640, 100]))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    again = step()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("topk", [0, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_trees_at_once_and_back_to_back(dtype, topk):
    """Calls on two streams that overlap, and calls in a row whose inputs the
    kernel before them has just written: the same bits as one at a time."""
    B, Hq, Hkv, d, T, N = 2, 8, 2, 128, 24, 2048
    xs = [S.tree_case(50 + i, B, Hq, Hkv, d, T, N, [2000 - 31 * i, 700 + i], max(topk, 1), dtype,
                      "f32", "tree") for i in range(2)]
    sets = []
    for x in xs:
        t = {n: x[n + "_t"].to(DEV) for n in ("q", "kd", "vd", "kc", "vc", "ksum")}
        t.update(lens=i32(x["lens"]), par=i32(x["parents"]))
        sets.append(t)

    def call(t, stream=None, q=None):
        return sas.sas_decode_tree(t["q"] if q is None else q, t["kd"], t["vd"], t["kc"], t["vc"],
                                   t["lens"], t["ksum"], topk, parents=t["par"], stream=stream)
    want = [call(t) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[call(t, s) for _ in range(30)] for t, s in zip(sets, streams) for _ in range(1)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(o, w) for o in g)
    # the output of one call is the next one's query, and lengths change in place
    chain, lens = [sets[0]["q"]], sets[0]["lens"]
    seq = []
    for i in range(6):
        chain.append(call(sets[0], q=chain[-1]))
        lens.sub_(64)
    torch.cuda.synchronize()
    lens.copy_(i32(xs[0]["lens"]))
    for i in range(6):
        torch.cuda.synchronize()
        assert torch.equal(call(sets[0], q=chain[i]), chain[i + 1])
        lens.sub_(64)
        torch.cuda.synchronize()


def test_caches_past_two_billion_elements():
    """Three sequences of 2^20 - 40 tokens, 8 kv heads of 128: element offsets
    pass 2^31. The last sequence against a call on a copy of its own (other
    splits: the tree's bound twice), and tokens written at its end."""
    B, Hq, Hkv, d, T, N, topk = 3, 8, 8, 128, 4, 1 << 20, 2
    g = torch.Generator(device=DEV).manual_seed(1)
    kc = torch.zeros((B, Hkv, N, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    assert kc.numel() > 1 << 31
    ks = torch.zeros((B, Hkv, N // 64, d), device=DEV)
    n = N - 40
    q = torch.randn((B, Hq, T, d), generator=g, device=DEV).bfloat16()
    kd = torch.randn((B, Hkv, T, d), generator=g, device=DEV).bfloat16()
    vd = torch.randn((B, Hkv, T, d), generator=g, device=DEV).bfloat16()
    for m in (5, N // 64 - 3):  # two blocks that score, and the tail
        kc[:, :, 64 * m:64 * m + 64] = torch.randn((B, Hkv, 64, d), generator=g, device=DEV).bfloat16()
        vc[:, :, 64 * m:64 * m + 64] = torch.randn((B, Hkv, 64, d), generator=g, device=DEV).bfloat16()
        ks[:, :, m] = 3.0 * q[:, :, 0].float()
    vc[:, :, N - 64:n] = 1.0
    lens = i32([n] * B)
    idx = torch.empty((B, Hkv, T, topk), dtype=torch.int32, device=DEV)
    o = sas.sas_decode_tree(q, kd, vd, kc, vc, lens, ks, topk, idx_out=idx)
    own = [t[2:].clone() for t in (q, kd, vd, kc, vc, ks)]
    one = sas.sas_decode_tree(own[0], own[1], own[2], own[3], own[4], lens[2:].clone(), own[5], topk)
    assert (idx[:, :, 0] == torch.tensor([5, N // 64 - 3], device=DEV)).all()
    err = (o[2:].float() - one.float()).abs().max()
    # weights and outputs round to bf16 on both sides; |v| < 5.5
    assert err <= 2 * 2 * 2.0 ** -8 * 5.5
    table = torch.arange(B * N // 64, dtype=torch.int32, device=DEV).view(B, -1)
    pools = [t.view(B, Hkv, N // 64, 64, d)[2:].transpose(1, 2).reshape(-1, Hkv, 64, d).contiguous()
             for t in (kc, vc)]
    sas.sas_cache_append(kd, vd, lens, kc, vc, ksum=ks)
    assert torch.equal(kc[2, :, n:n + T], kd[2]) and torch.equal(vc[2, :, n:n + T], vd[2])
    assert (kc[:, :, n + T:] == 0).all() and (kc[0, :, N - 64:n] == 0).all()
    paged = sas.sas_decode_tree(own[0], own[1], own[2], pools[0], pools[1], lens[2:].clone(),
                                own[5][0].transpose(0, 1).contiguous(), topk,
                                block_table=table[:1].clone())
    assert torch.equal(paged, one)
    del kc, vc, own, pools
    torch.cuda.empty_cache()


def test_decode_tree_defaults_are_a_full_chain():
    x = S.tree_case(12, 2, 4, 2, 64, 9, 640, [600, 0], 3, "bf16", "f32", "chain")
    a = tree_call(x, 3, 1, False)
    t = {n: x[n + "_t"].to(DEV) for n in ("q", "kd", "vd", "kc", "vc", "ksum")}
    b = sas.sas_decode_tree(t["q"], t["kd"], t["vd"], t["kc"], t["vc"], i32(x["lens"]), t["ksum"],
                            3, ws=torch.empty(1 << 22, dtype=torch.uint8, device=DEV))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,paged", [("bf16", True), ("f32", False)])
def test_speculative_serving_steps(dtype, paged):
    """Prompt, then rounds of draft, tree decode, acceptance, page map and
    cache write, against the oracle on caches kept on the host; at the end one
    plain decode step over what the rounds have built."""
    B, Hq, Hkv, d, T, topk, width = 2, 4, 2, 64, 16, 3, 8
    rng = np.random.Generator(np.random.PCG64(77))
    f, amp = rope.inv_freq(d, scaling="linear", factor=2.0)
    fd, f64 = f.to(DEV), f.double().numpy()
    N = 64 * width
    npages = B * width + 1
    shape = (npages, Hkv, 64, d) if paged else (B, Hkv, N, d)
    dt = S.TORCH[dtype]
    kc = torch.full(shape, float("nan"), dtype=dt, device=DEV)
    vc = torch.full(shape, float("nan"), dtype=dt, device=DEV)
    ks = torch.full((npages, Hkv, d) if paged else (B, Hkv, width, d), float("nan"), device=DEV)
    table = i32(np.full((B, width), -1))
    free, head = i32(rng.permutation(npages)), i32([0])
    lens = i32([0, 0])

    def write(k, v, n, rows=None, inv=None):
        nn = i32(n)
        slots, new, taken, h = sas.sas_page_map(lens, nn, table, free, head, k.shape[2], npages,
                                                out=None)
        assert (taken >= 0).all()
        sas.sas_cache_append(k, v, lens, kc, vc, ksum=ks, ntok=nn, rows=rows,
                             slots=slots if paged else None, inv_freq=inv)
        lens.copy_(new)
        head.copy_(h)

    def gathered():
        if not paged:
            return np64(kc), np64(vc), np64(ks)
        at = table.long().clamp(min=0)
        return (np64(kc[at].transpose(1, 2).reshape(B, Hkv, N, d)),
                np64(vc[at].transpose(1, 2).reshape(B, Hkv, N, d)),
                np64(ks[at].transpose(1, 2)))
    prompt = [150, 61]
    # block means spread along one direction that the queries share
    w = rng.standard_normal((Hkv, d))
    w /= np.linalg.norm(w, axis=1, keepdims=True)

    def keys(n):
        lev = rng.standard_normal((B, 1, n, 1)) * 0.5
        return rng.standard_normal((B, Hkv, n, d)) + 8.0 * lev * w[None, :, None]
    dev = lambda a: S.rounded(a, dtype)[0].reshape(a.shape).to(DEV)
    write(dev(keys(150)), dev(rng.standard_normal((B, Hkv, 150, d))), prompt, inv=fd)
    for step in range(4):
        par = S.parents_of("tree", B, T, rng)
        q = dev(rng.standard_normal((B, Hq, T, d)) * 2)
        k, v = dev(keys(T)), dev(rng.standard_normal((B, Hkv, T, d)))
        qr, kr = sas.sas_rotary(q, fd, k=k, start=lens, parents=i32(par))
        o = sas.sas_decode_tree(qr, kr, v, kc, vc, lens, ks, topk, parents=i32(par),
                                block_table=table if paged else None)
        hk, hv, hs = gathered()
        x = dict(q=np64(qr), kd=np64(kr), vd=np64(v), kc=np.nan_to_num(hk), vc=np.nan_to_num(hv))
        ref, _, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], hk, hv, lens.tolist(), hs, par,
                                      [T] * B, topk)
        assert (np.abs(np64(o) - ref) <= tree_tol(x, ref, mass, topk, dtype, "f32")).all()
        # accept one path of each sequence, already rotated
        rows, n = np.zeros((B, T), dtype=np.int32), []
        for b in range(B):
            path = [int(rng.integers(4, T))]
            while par[b, path[0]] >= 0:
                path.insert(0, int(par[b, path[0]]))
            rows[b, :len(path)] = path
            n.append(len(path))
        write(kr, v, n, rows=i32(rows))
    hk, hv, hs = gathered()
    for b in range(B):
        L = int(lens[b])
        assert np.isfinite(hk[b, :, :L]).all() and np.isfinite(hs[b, :, :L // 64]).all()
        mean = hk[b, :, :L // 64 * 64].reshape(Hkv, -1, 64, d).mean(2)
        assert np.abs(mean - hs[b, :, :L // 64]).max() <= 64 * U * np.nanmax(np.abs(hk)) * 2
    q = dev(rng.standard_normal((B, Hq, 1, d)))
    k, v = dev(keys(1)), dev(rng.standard_normal((B, Hkv, 1, d)))
    slots, new, _, _ = sas.sas_page_map(lens, i32([1, 1]), table, free, head, 1, npages)
    qr = sas.sas_cache_append(k, v, lens, kc, vc, ksum=ks, slots=slots if paged else None,
                              inv_freq=fd, q=q)
    pos = lens.cpu().numpy()[:, None]
    assert (np.abs(np64(qr) - SO.rotate(np64(q), pos, f64)) <=
            rot_tol(np64(q), SO.rotate(np64(q), pos, f64), d, False, 1.0, dtype)).all()
    # cached rows past the end may hold anything the caches were made of
    kc2, vc2, ks2 = (torch.nan_to_num(t) for t in (kc, vc, ks))
    step_q = qr[:, :, 0].contiguous()
    if paged:
        o = sas.sas_decode_paged(step_q, kc2, vc2, ks2, table.clamp(min=0), new, topk)
    else:
        o = sas.sas_decode(step_q, kc2, vc2, new, ks2, topk)
    hk, hv, hs = gathered()
    x = dict(q=np64(qr), kd=np.zeros((B, Hkv, 1, d)), vd=None, kc=np.nan_to_num(hk))
    from oracle import sas_oracle as O
    sel, cnt, logg, _ = O.select_decode(np64(step_q), hs, new.tolist(), Hkv, topk)
    ref, _ = O.decode_attend(np64(step_q), hk, hv, new.tolist(), sel, cnt, logg, Hkv)
    mass, _ = O.decode_attend(np64(step_q), hk, np.abs(hv), new.tolist(), sel, cnt, logg, Hkv)
    tol = tree_tol(x, ref[:, :, None], mass[:, :, None], topk, dtype, "f32")[:, :, 0]
    assert (np.abs(np64(o) - ref) <= tol).all()
