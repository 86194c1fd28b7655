"""Seeded inputs of the serving tests (host, numpy): drafted trees over caches
whose block scores are planted, so that the Top-K order is decided by far more
than fp32 rounding (levels 0.03 apart)."""
import numpy as np
import torch

from gated_block_sparse_b200 import inputs

BLOCK = 64
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def rounded(x, dtype):
    """fp64 values after one rounding to dtype, as (tensor, fp64 array)."""
    t = inputs.to_storage(np.asarray(x, dtype=np.float64), dtype)
    return t, t.double().numpy()


def store(dtype):
    return lambda x: rounded(x, dtype)[1].reshape(np.shape(x))


def parents_of(kind, B, T, rng):
    if kind == "chain":
        return np.tile(np.arange(T, dtype=np.int32) - 1, (B, 1))
    p = np.full((B, T), -1, dtype=np.int32)
    if kind == "tree":
        for b in range(B):
            for i in range(1, T):
                p[b, i] = max(-1, i - int(rng.integers(1, 4)))
    return p  # "flat": every token a root


def tree_case(seed, B, Hq, Hkv, d, T, N, lens, topk, dtype, sums, kind, ntok=None):
    """Contiguous inputs as fp64 arrays, already rounded to their types."""
    rng = np.random.Generator(np.random.PCG64(seed))
    G, C = Hq // Hkv, N // BLOCK
    scale, kappa, topics = 1.0 / np.sqrt(d), 6.0, 2
    kc = rng.standard_normal((B, Hkv, C, BLOCK, d))
    vc = rng.standard_normal((B, Hkv, N, d))
    q = rng.standard_normal((B, Hkv, G, T, d))
    kd = rng.standard_normal((B, Hkv, T, d))
    vd = rng.standard_normal((B, Hkv, T, d))
    for b in range(B):
        topic = rng.integers(0, topics, T)
        for r in range(Hkv):
            w = np.linalg.qr(rng.standard_normal((d, topics)))[0]
            level = np.stack([0.03 * rng.permutation(C) for _ in range(topics)])
            kc[b, r] -= kc[b, r].mean(1, keepdims=True)
            kc[b, r] += (level.T @ w.T / (scale * kappa))[:, None]
            q[b, r] += (kappa * w.T[topic] - (q[b, r] @ w) @ w.T)
            # drafted keys near the middle of the levels, between two of them
            kd[b, r] += 0.03 * (C // 2 + 0.5) / (scale * kappa) * w.sum(1)
    par = parents_of(kind, B, T, rng)
    ntok = [T] * B if ntok is None else ntok
    x = dict(q=q.reshape(B, Hq, T, d), kd=kd, vd=vd, kc=kc.reshape(B, Hkv, N, d), vc=vc)
    out = {}
    for n, v in x.items():
        out[n + "_t"], out[n] = rounded(v, dtype)
        out[n] = out[n].reshape(v.shape)
        out[n + "_t"] = out[n + "_t"].reshape(v.shape)
    mean = out["kc"].reshape(B, Hkv, C, BLOCK, d).mean(3)
    out["ksum_t"], out["ksum"] = rounded(mean, sums)
    out["ksum_t"] = out["ksum_t"].reshape(mean.shape)
    out["ksum"] = out["ksum"].reshape(mean.shape)
    out.update(lens=np.array(lens, dtype=np.int32), ntok=np.array(ntok, dtype=np.int32),
               parents=par, rng=rng)
    return out


def to_pages(x, rng, spare=3):
    """The contiguous caches of a case as pools of shuffled pages: (kpool,
    vpool, kspool, table) tensors; pages that no table names hold NaN."""
    B, Hkv, N, d = x["kc_t"].shape
    C = N // BLOCK
    perm = rng.permutation(B * C + spare)[:B * C].reshape(B, C)
    pools = []
    for n in ("kc_t", "vc_t"):
        t = torch.full((B * C + spare, Hkv, BLOCK, d), float("nan"), dtype=x[n].dtype)
        t[torch.from_numpy(perm)] = x[n].reshape(B, Hkv, C, BLOCK, d).transpose(1, 2)
        pools.append(t)
    ks = torch.full((B * C + spare, Hkv, d), float("nan"), dtype=x["ksum_t"].dtype)
    ks[torch.from_numpy(perm)] = x["ksum_t"].transpose(1, 2)
    return pools[0], pools[1], ks, torch.from_numpy(perm.astype(np.int32))
