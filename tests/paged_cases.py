"""Inputs of the paged operators' tests: ragged batches over shuffled pages, whose unused pages and
slots hold NaN, and the tolerances that follow from the kernels' roundings."""
import numpy as np
import torch

from tests import parity

E4M3 = torch.float8_e4m3fn


def to_cache(x, scale, e4m3):
    return (x / scale).clamp(-448, 448).to(E4M3) if e4m3 else x.to(torch.bfloat16)


def make(new, keys, H_q, H_kv, D, page, e4m3=False, seed=0, extra_rows=0, spare_pages=2, max_pages=None, q_gain=1.0,
         poison=True):
    """A batch of sequences with ``new[b]`` new tokens and ``keys[b]`` keys (CPU tensors)."""
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    need = [-(-k // page) for k in keys]
    n_pages = sum(need) + spare_pages
    width = max(max(need), 1) if max_pages is None else max_pages
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((B, width), 2 ** 30, dtype=torch.int32)  # entries past a sequence's pages are never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    k = torch.randn((n_pages, page, H_kv, D), generator=g)
    v = torch.randn((n_pages, page, H_kv, D), generator=g)
    k_scale, v_scale = (0.03125, 0.02) if e4m3 else (1.0, 1.0)
    kc, vc = to_cache(k, k_scale, e4m3), to_cache(v, v_scale, e4m3)
    if poison:
        used = torch.zeros((n_pages, page), dtype=torch.bool)
        for b in range(B):
            for j in range(need[b]):
                used[table[b, j], : min(page, keys[b] - j * page)] = True
        bits = kc.view(torch.uint8 if e4m3 else torch.int16), vc.view(torch.uint8 if e4m3 else torch.int16)
        for x in bits:
            x[~used] = 0x7F if e4m3 else 0x7FC0  # NaN
    T = sum(new) + extra_rows
    q = (torch.randn((T, H_q, D), generator=g) * q_gain).to(torch.bfloat16)
    start = np.concatenate([[0], np.cumsum(new)]).astype(int)
    return {"q": q, "k_cache": kc, "v_cache": vc, "page_table": table,
            "seq_len": torch.tensor(keys, dtype=torch.int32), "q_start": torch.tensor(start, dtype=torch.int32),
            "k_scale": k_scale, "v_scale": v_scale, "new": list(new), "keys": list(keys), "start": start.tolist()}


def to_gpu(x):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def handle(attn, g):
    return attn.PagedKV(g["k_cache"], g["v_cache"], g["page_table"], g["seq_len"], g["q_start"],
                        k_scale=g["k_scale"], v_scale=g["v_scale"])


def check_attend(o, lse, want, rows, what="", e4m3=False, score_error=0.0):
    """o and lse against the oracle's (o, lse, a) on the given token rows.

    o: the output's rounding (half a bf16 step: 2^-8 relative), each softmax weight's rounding to bf16, or
    to two e4m3 terms whose sum is as exact (2^-8 relative to the weight: at most 2^-8 a, a = P |V|), and 2^-12 a for
    what is computed in fp32 (the scores' sums, below 5.5e-5 as the next lines say; ex2 is within 2^-22).
    e4m3 terms step by 2^-9 at the least, so a small weight is off by up to 2^-10; the kernels keep a row's
    largest weight at 2^7 or more: 2^-17 of the largest weight for each key, 2^-17 f together.
    lse: the fp32 sums of 128 products that make a score, 128 x 2^-24 x sum |q k| scale, below 5.5e-5 for normal
    inputs, and the row's own sum (some 25 terms' roundings of 2^-24); 6e-5 holds both.  score_error: what the scores' fp32 sums may be off by for larger inputs; it
    joins lse's bound, and twice it (a weight's numerator and the sum) times a joins o's."""
    o_ref, lse_ref, a, f = want
    o, lse = parity.to_np(o)[rows], parity.to_np(lse)[:, rows]
    o_ref, a, f, lse_ref = o_ref[rows], a[rows], f[rows], lse_ref[:, rows]
    assert np.all(np.isfinite(o)), f"{what}: non-finite O"
    err = np.abs(o - o_ref)
    bound = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -8 + 2.0 ** -12) * a + (2.0 ** -17 * f if e4m3 else 0.0) + 2 * score_error * a + 1e-30
    worst = np.argmax(err - bound)
    assert np.all(err <= bound), f"{what}: O error {err.flat[worst]:.3e} > bound {bound.flat[worst]:.3e}"
    # taken together the errors are independent: the root mean square is well below the bound's
    assert np.sqrt(np.mean(err ** 2)) <= (2.0 ** -8 + score_error) * np.sqrt(np.mean(a ** 2)) + 1e-30, f"{what}: O rms"
    inf = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), inf), f"{what}: -inf pattern of lse differs"
    assert np.all(np.abs(lse[~inf] - lse_ref[~inf]) <= 6e-5 + score_error), f"{what}: lse {np.abs(lse[~inf] - lse_ref[~inf]).max():.3e}"
