"""The serving calls without a GPU: the C ABI's refusals, the binding's checks,
the frequencies, and pins of the serving oracle (CPU only: no call here reaches
a kernel)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import serving_cases as S
from gated_block_sparse_b200 import rope, sas
from oracle import serving_oracle as SO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from gated_block_sparse_b200 import build
    build.build()
    return sas.load_library()


def test_every_declared_symbol_is_exported(lib):
    src = open(os.path.join(ROOT, "include", "sas_serving.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(sas_[a-z_0-9]+)\s*\(", src)))
    assert names == ["sas_cache_append", "sas_decode_tree", "sas_decode_tree_workspace_size",
                     "sas_page_map", "sas_rotary"]
    for n in names:
        assert hasattr(lib, n) and n in sas.SIGNATURES


ROTARY = dict(q=FAKE, qs=None, qo=FAKE, qos=None, Hq=4, k=FAKE, ks=None, ko=FAKE, kos=None, Hkv=2,
              dt=1, B=1, N=8, d=128, f=FAKE, rot=128, inter=0, amp=1.0, inverse=0, pos=None,
              start=None, parents=None, stream=None)
PAGES = dict(lens=FAKE, nnew=FAKE, table=FAKE, free=FAKE, head=FAKE, B=2, T=4, width=3, npages=10,
             nfree=4, slots=FAKE, new=FAKE, taken=FAKE, out=FAKE, stream=None)
APPEND = dict(q=None, qs=None, qo=None, k=FAKE, ks=None, v=FAKE, vs=None, dt=1, B=1, Hq=4, Hkv=2,
              T=4, d=128, rows=None, lens=FAKE, ntok=None, f=None, rot=0, inter=0, amp=1.0,
              slots=None, kc=FAKE, vc=FAKE, N=128, npages=0, ksum=FAKE, sdt=0, stream=None)
TREE = dict(q=FAKE, kd=FAKE, vd=FAKE, kc=FAKE, vc=FAKE, dt=1, B=1, Hq=4, Hkv=2, T=4, N=128, d=128,
            parents=None, ntok=None, lens=FAKE, ksum=FAKE, sdt=0, table=None, npages=0, topk=2,
            gated=1, scale=0.0, o=FAKE, idx=None, ws=FAKE, nws=BIG, stream=None)


def stride(*s):
    return (ctypes.c_int64 * 3)(*s)


@pytest.mark.parametrize("fn,base,change,status,text", [
    ("sas_rotary", ROTARY, dict(d=96), 2, b"head dim"),
    ("sas_rotary", ROTARY, dict(dt=2), 1, b"dtype"),
    ("sas_rotary", ROTARY, dict(rot=130), 1, b"rot must be even"),
    ("sas_rotary", ROTARY, dict(rot=0), 1, b"rot must be even"),
    ("sas_rotary", ROTARY, dict(rot=7), 1, b"rot must be even"),
    ("sas_rotary", ROTARY, dict(q=None), 1, b"q must not be NULL"),
    ("sas_rotary", ROTARY, dict(qo=FAKE + 8), 1, b"qo must be 16-byte aligned"),
    ("sas_rotary", ROTARY, dict(k=None), 1, b"k goes with"),
    ("sas_rotary", ROTARY, dict(ko=None), 1, b"ko must not be NULL"),
    ("sas_rotary", ROTARY, dict(amp=float("nan")), 1, b"amplitude"),
    ("sas_rotary", ROTARY, dict(inter=2), 1, b"interleaved"),
    ("sas_rotary", ROTARY, dict(inverse=3), 1, b"inverse"),
    ("sas_rotary", ROTARY, dict(pos=FAKE, start=FAKE), 1, b"excludes"),
    ("sas_rotary", ROTARY, dict(start=FAKE + 4), 1, b"start"),
    ("sas_rotary", ROTARY, dict(B=70000), 2, b"65535"),
    ("sas_rotary", ROTARY, dict(qs=stride(0, -128, 128)), 1, b"input strides"),
    ("sas_rotary", ROTARY, dict(kos=stride(2048, 1024, 64)), 1, b"output strides"),
    ("sas_rotary", ROTARY, dict(qos=stride(4096, 0, 128)), 1, b"output strides"),
    ("sas_page_map", PAGES, dict(B=-1), 1, b"sizes"),
    ("sas_page_map", PAGES, dict(npages=1 << 26), 2, b"npages"),
    ("sas_page_map", PAGES, dict(B=60000, T=1 << 20), 2, b"2^31"),
    ("sas_page_map", PAGES, dict(width=1 << 26), 2, b"width"),
    ("sas_page_map", PAGES, dict(slots=None), 1, b"slots"),
    ("sas_page_map", PAGES, dict(head=None), 1, b"free_head"),
    ("sas_page_map", PAGES, dict(table=FAKE + 4), 1, b"block_table"),
    ("sas_cache_append", APPEND, dict(d=80), 2, b"head dim"),
    ("sas_cache_append", APPEND, dict(N=100), 1, b"multiple of 64"),
    ("sas_cache_append", APPEND, dict(slots=FAKE), 1, b"npages"),
    ("sas_cache_append", APPEND, dict(q=FAKE, qo=FAKE), 1, b"inv_freq"),
    ("sas_cache_append", APPEND, dict(q=FAKE, qo=FAKE, f=FAKE, rot=64, rows=FAKE), 1, b"rows"),
    ("sas_cache_append", APPEND, dict(q=FAKE, qo=None, f=FAKE, rot=64), 1, b"qo"),
    ("sas_cache_append", APPEND, dict(f=FAKE, rot=200), 1, b"rot"),
    ("sas_cache_append", APPEND, dict(sdt=5), 1, b"summary dtype"),
    ("sas_cache_append", APPEND, dict(lens=None), 1, b"lens"),
    ("sas_cache_append", APPEND, dict(vs=stride(1, -1, 1)), 1, b"input strides"),
    ("sas_cache_append", APPEND, dict(kc=FAKE + 2), 1, b"kc"),
    ("sas_decode_tree", TREE, dict(T=65), 2, b"64 drafted"),
    ("sas_decode_tree", TREE, dict(T=0), 1, b"T must be"),
    ("sas_decode_tree", TREE, dict(N=100), 1, b"multiple of 64"),
    ("sas_decode_tree", TREE, dict(N=0), 1, b"multiple of 64"),
    ("sas_decode_tree", TREE, dict(N=(1 << 20) + 64), 2, b"2^20"),
    ("sas_decode_tree", TREE, dict(Hq=18), 2, b"query heads"),
    ("sas_decode_tree", TREE, dict(Hq=5), 1, b"multiple"),
    ("sas_decode_tree", TREE, dict(topk=129), 2, b"topk"),
    ("sas_decode_tree", TREE, dict(gated=2), 1, b"gated"),
    ("sas_decode_tree", TREE, dict(sdt=9), 1, b"summary dtype"),
    ("sas_decode_tree", TREE, dict(table=FAKE), 1, b"npages"),
    ("sas_decode_tree", TREE, dict(ksum=None), 1, b"ksum"),
    ("sas_decode_tree", TREE, dict(parents=FAKE + 4), 1, b"parents"),
    ("sas_decode_tree", TREE, dict(ws=None), 1, b"ws must not be NULL"),
    ("sas_decode_tree", TREE, dict(nws=16), 1, b"workspace too small"),
])
def test_refusals(lib, fn, base, change, status, text):
    st = getattr(lib, fn)(*{**base, **change}.values())
    assert st == status and text in lib.sas_last_error_message(), lib.sas_last_error_message()


@pytest.mark.parametrize("fn,base,change,status,text", [
    ("sas_rotary", ROTARY, dict(parents=FAKE, N=1025), 2, b"1024 with parents"),
    ("sas_cache_append", APPEND, dict(T=(1 << 30) + 1, ks=stride(0, 128, 0), vs=stride(0, 128, 0)),
     2, b"2^30"),
])
def test_refusals_of_sizes(lib, fn, base, change, status, text):
    test_refusals(lib, fn, base, change, status, text)


@pytest.mark.parametrize("change,text", [
    # B 2, N 8, d 128, bf16: contiguous q [2][4][8][128], 16384 bytes; k half of it
    (dict(qos=stride(4096, 128, 128)), b"output rows must not overlap"),
    (dict(qos=stride(1024, 1024, 128)), b"output rows must not overlap"),
    (dict(kos=stride(2048, 1024, 1024)), b"output rows must not overlap"),
    (dict(ko=FAKE + (2 << 20) + 16384 - 16), b"qo and ko"),
    (dict(qo=FAKE + (1 << 20), qos=stride(4096, 128, 512)), b"an output must be"),
    (dict(qo=FAKE + (1 << 20) + 256), b"an output must be"),
    (dict(qo=FAKE + (1 << 20) - 16368), b"an output must be"),
    (dict(qo=FAKE + (3 << 20)), b"an output must be"),  # k
    # views of one buffer [2][8][6 heads][128]: k's heads into q's, or a token ahead
    (dict(qs=stride(6144, 128, 768), ks=stride(6144, 128, 768), k=FAKE + (1 << 20) + 1024,
          kos=stride(6144, 128, 768), ko=FAKE + (1 << 20) + 768), b"an output must be"),
    (dict(qs=stride(6144, 128, 768), qo=FAKE + (1 << 20) + 1536, qos=stride(6144, 128, 768)),
     b"an output must be"),
])
def test_rotary_refuses_memory_that_overlaps(lib, change, text):
    base = dict(ROTARY, B=2, q=FAKE + (1 << 20), qo=FAKE + (2 << 20), k=FAKE + (3 << 20),
                ko=FAKE + (4 << 20))
    st = lib.sas_rotary(*{**base, **change}.values())
    assert st == 1 and text in lib.sas_last_error_message(), lib.sas_last_error_message()


@pytest.mark.parametrize("change,text", [
    # k and v are [1][2][4][128] bf16, 2048 bytes; a cache is [1][2][128][128], 65536
    (dict(vc=FAKE + (2 << 20)), b"kc and vc"),
    (dict(vc=FAKE + (2 << 20) + 65520), b"kc and vc"),
    (dict(k=FAKE + (2 << 20) + 65520), b"k and v must not lie"),
    (dict(v=FAKE + (3 << 20) - 16), b"k and v must not lie"),
    (dict(k=FAKE + (2 << 20) - 1008, ks=stride(0, 0, 128)), b"k and v must not lie"),
    (dict(slots=FAKE, npages=5, N=0, k=FAKE + (2 << 20) + 5 * 32768 - 16), b"k and v must not lie"),
    (dict(qo=FAKE + (4 << 20) + 16), b"qo must be q itself"),
    (dict(qo=FAKE + (4 << 20), qs=stride(0, 128, 512)), b"qo must be q itself"),
    (dict(qo=FAKE + (2 << 20) + 128), b"qo must lie apart"),
    (dict(qo=FAKE + (5 << 20)), b"qo must lie apart"),
])
def test_append_refuses_memory_that_overlaps(lib, change, text):
    base = dict(APPEND, q=FAKE + (4 << 20), qo=FAKE + (6 << 20), f=FAKE, rot=64,
                k=FAKE + (1 << 20), v=FAKE + (5 << 20), kc=FAKE + (2 << 20), vc=FAKE + (3 << 20))
    st = lib.sas_cache_append(*{**base, **change}.values())
    assert st == 1 and text in lib.sas_last_error_message(), lib.sas_last_error_message()


@pytest.mark.parametrize("change,text", [
    # B 2, T 4, width 3, nfree 4: slots 32 bytes, table 24, free list 16, the rest 8 and 4
    (dict(new="nnew"), b"new_lens and nnew"),
    (dict(new=0x20000 + 0), b"new_lens and slots"),
    (dict(taken="lens"), b"taken and lens"),
    (dict(taken="new"), b"new_lens and taken"),
    (dict(out="taken"), b"taken and head_out"),
    (dict(slots="free"), b"slots and free_pages"),
    (dict(slots=0x60000 - 16), b"slots and free_pages"),
    (dict(table=0x50000 - 16), b"block_table and nnew"),
    (dict(out="free"), b"head_out and free_pages"),
    (dict(new=0x40000 + 0, out="head", taken=0x70000), b"taken and head_out"),
])
def test_page_map_refuses_memory_that_overlaps(lib, change, text):
    base = dict(PAGES, slots=0x20000, table=0x30000, lens=0x40000, nnew=0x50000, free=0x60000,
                head=0x70000, new=0x80000, taken=0x90000, out=0xA0000)
    change = {k: base[v] if isinstance(v, str) else v for k, v in change.items()}
    st = lib.sas_page_map(*{**base, **change}.values())
    names = text.split(b" and ")
    assert st == 1 and all(n in lib.sas_last_error_message() for n in names), \
        lib.sas_last_error_message()


def test_empty_calls_need_no_pointers(lib):
    none = dict.fromkeys(["q", "qo", "k", "ko", "f"], None)
    assert lib.sas_rotary(*{**ROTARY, **none, "Hkv": 0, "B": 0}.values()) == 0
    assert lib.sas_cache_append(*{**APPEND, "k": None, "lens": None, "T": 0}.values()) == 0
    assert lib.sas_decode_tree(*{**TREE, "q": None, "ws": None, "B": 0}.values()) == 0


def test_tree_workspace_grows_with_the_problem(lib):
    size = lib.sas_decode_tree_workspace_size
    a = size(1, 32, 8, 4, 65536, 128, 15, 1)
    assert 0 < a < size(8, 32, 8, 16, 131072, 128, 31, 1)
    assert size(1, 32, 8, 4, 65536, 128, 0, 1) < a  # no selection: partial outputs only
    assert size(1, 32, 8, 65, 65536, 128, 15, 1) == 0 and size(0, 32, 8, 4, 65536, 128, 15, 1) == 0


def test_binding_wants_cuda_tensors_of_the_right_kind():
    q, f = torch.zeros(1, 2, 4, 64), torch.zeros(16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        sas.sas_rotary(q, f)
    with pytest.raises(ValueError, match="CUDA device"):
        sas.sas_page_map(i, i, i.view(1, 1), i, i, 1, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        sas.sas_cache_append(q, q, i, q, q)
    with pytest.raises(ValueError, match="CUDA device"):
        sas.sas_decode_tree(q, q, q, q, q, i, None, 0)


def test_inverse_frequencies():
    f, a = rope.inv_freq(128)
    assert f.dtype == torch.float32 and f.shape == (64,) and a == 1.0
    assert f[0] == 1.0 and abs(float(f[32]) - 1e-2) < 1e-9
    lin, _ = rope.inv_freq(128, scaling="linear", factor=4.0)
    assert torch.equal(lin, f / 4)
    base, _ = rope.inv_freq(128, scaling="base", factor=4.0)
    assert base[0] == 1.0 and abs(float(base[-1] / f[-1]) - 0.25) < 1e-6
    parts, amp = rope.inv_freq(128, scaling="parts", factor=16.0, trained=8192)
    turns = 8192 * f / (2 * np.pi)
    assert torch.equal(parts[turns > 32.1], f[turns > 32.1])
    assert torch.allclose(parts[turns < 0.99], f[turns < 0.99] / 16)
    assert (parts <= f).all() and (parts * 16 >= f * (1 - 1e-6)).all()
    assert abs(amp - (1 + 0.1 * np.log(16.0))) < 1e-12
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, base=0.0),
                dict(rot=8, scaling="other"), dict(rot=8, scaling="parts", slow=2.0, fast=1.0)):
        with pytest.raises(ValueError):
            rope.inv_freq(**bad)


@pytest.mark.parametrize("bad", [
    dict(base=float("inf")), dict(base=float("nan")),
    dict(scaling="linear", factor=float("inf")),
    dict(scaling="parts", factor=2.0, trained=0),
    dict(scaling="parts", factor=2.0, trained=float("nan")),
    dict(scaling="parts", factor=2.0, fast=float("inf"))])
def test_inverse_frequencies_refuse_what_is_not_finite(bad):
    with pytest.raises(ValueError):
        rope.inv_freq(8, **bad)


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_rotation_is_a_complex_product(inter):
    rng = np.random.Generator(np.random.PCG64(0))
    x = rng.standard_normal((2, 3, 5, 16))
    pos = rng.integers(0, 10 ** 6, (2, 5))
    f = rng.random(6)
    y = SO.rotate(x, pos, f, inter, 1.5)
    a, b = (x[..., 0:12:2], x[..., 1:12:2]) if inter else (x[..., :6], x[..., 6:12])
    z = (a + 1j * b) * 1.5 * np.exp(1j * pos[:, None, :, None] * f)
    u, v = (y[..., 0:12:2], y[..., 1:12:2]) if inter else (y[..., :6], y[..., 6:12])
    assert np.abs(u - z.real).max() < 1e-12 and np.abs(v - z.imag).max() < 1e-12
    assert np.array_equal(y[..., 12:], x[..., 12:])
    back = SO.rotate(y, pos, f, inter, 1 / 1.5, inverse=True)
    assert np.abs(back - x).max() < 1e-12


def test_oracle_tree_is_dense_attention_when_every_block_is_kept():
    """topk >= C and gates left out: softmax over the cache and the path."""
    x = S.tree_case(3, 1, 2, 1, 64, 9, 256, [190], 8, "f32", "f32", "tree")
    o, idx, mass = SO.decode_tree(x["q"], x["kd"], x["vd"], x["kc"], x["vc"], x["lens"],
                                  x["ksum"], x["parents"], x["ntok"], 8, gated=0)
    assert SO.depths(x["parents"]).max() > 2  # some paths fill the tail's block
    for i in range(9):
        path = [i]
        while x["parents"][0, path[0]] >= 0:
            path.insert(0, int(x["parents"][0, path[0]]))
        k = np.concatenate([x["kc"][0, 0, :190], x["kd"][0, 0, path]])
        v = np.concatenate([x["vc"][0, 0, :190], x["vd"][0, 0, path]])
        z = x["q"][0, :, i] @ k.T / 8.0
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        assert np.abs(p @ v - o[0, :, i]).max() < 1e-12
        C = (190 + len(path) - 1) // 64
        assert idx[0, 0, i].tolist() == list(range(C)) + [-1] * (8 - C)
        assert (mass[0, :, i] >= np.abs(o[0, :, i]) - 1e-12).all()


def test_oracle_page_map_gives_each_token_its_own_slot():
    lens, nnew = [0, 63, 64, 130], [65, 1, 0, 64]
    table = np.full((4, 5), -1)
    free = np.arange(20, 40)
    table[1, 0], table[2, 0], table[3, :3] = 0, 1, [2, 3, 4]
    slots, new, taken, head, table = SO.page_map(lens, nnew, table, free, 2, 65, 50)
    assert new.tolist() == [65, 64, 64, 194] and taken.tolist() == [2, 0, 0, 1] and head == 5
    assert table[0, :2].tolist() == [22, 23] and table[3, 3] == 24
    used = slots[slots >= 0]
    assert len(set(used.tolist())) == 65 + 1 + 64
    assert slots[1, 0] == 63 and slots[3, 0] == 4 * 64 + 2 and slots[3, 62] == 24 * 64
