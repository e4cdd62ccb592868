"""Attention over a paged cache where one key stands far above thousands of others.

The many small weights then make up a share of the result that none of them shows by itself, so a floor under
the weights (small ones rounded to zero in P V, but not in the row's sum) shows as an error of one sign.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
PAGE = 1024


def _attn():
    import attention_attn_fwd_10_b200 as attn

    return attn


def _batch(n_seq, keys, H_q, H_kv, D, gap, e4m3, new=1, seed=0):
    """n_seq sequences of the same pages, each with ``new`` tokens of their own.  Key 5's score is `gap` nats
    above those of the others (normal, standard deviation 0.5), its value is small; the other values have a mean per channel."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    n_pages = -(-keys // PAGE)
    k, v = 0.5 * normal(n_pages * PAGE, H_kv, D), normal(n_pages * PAGE, H_kv, D) + 0.5 * normal(H_kv, D)
    q = normal(n_seq * new, H_q, D)
    q[..., 0] = 4.0
    k[..., 0] = 0.0
    k[5] = 0.0
    k[5, :, 0] = gap * math.sqrt(D) / 4.0
    v[5] *= 0.02
    k_scale, v_scale = (0.125, 0.02) if e4m3 else (1.0, 1.0)

    def cache(x, scale):
        x = x.view(n_pages, PAGE, H_kv, D)
        return (x / scale).clamp(-448, 448).to(E4M3) if e4m3 else x.bfloat16()

    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").expand(n_seq, n_pages).contiguous()
    lens = torch.full((n_seq,), keys, dtype=torch.int32, device="cuda")
    start = torch.arange(n_seq + 1, dtype=torch.int32, device="cuda") * new
    kc, vc = cache(k, k_scale), cache(v, v_scale)
    return q.bfloat16(), _attn().PagedKV(kc, vc, table, lens, start, k_scale=k_scale, v_scale=v_scale)


def _check(n_seq, keys, H_q, H_kv, D, gap, e4m3, hint, new=1):
    """o and lse against 64 bits, not causal.

    Bounds: half a bf16 step of the output (2^-8); each weight's own rounding, bf16 (2^-8) or, over an e4m3 cache,
    fp16 (2^-11), of a = P |V|; fp16 weights below its normal numbers step by 2^-24, and a row's largest stands at 2^7 or
    more: 2^-32 of the largest for each key, 2^-32 f with f = max P x sum |V|.  Scores: fp32 sums of D products,
    D x 2^-24 x sum |q k| scale; that joins lse's bound, and twice it times a o's; 2^-12 a and 6e-5 for the rest in fp32
    (ex2, the row's sum, the join of the pieces)."""
    q, cache = _batch(n_seq, keys, H_q, H_kv, D, gap, e4m3, new)
    o, lse = _attn().fwd_paged(cache, q, causal=False, max_new=hint)
    torch.cuda.synchronize()
    assert _attn().device_status() == 0
    scale, G = D ** -0.5, H_q // H_kv
    step = 2.0 ** -11 if e4m3 else 2.0 ** -8
    for h in range(H_q):
        k = cache.k.float().double().flatten(0, 1)[:keys, h // G] * cache.k_scale
        v = cache.v.float().double().flatten(0, 1)[:keys, h // G] * cache.v_scale
        for r in range(0, n_seq * new, 64):
            x = q[r:r + 64, h].double()
            s = x @ k.T * scale
            score_error = D * 2.0 ** -24 * float((x.abs() @ k.abs().T).max()) * scale
            want_lse = torch.logsumexp(s, -1)
            p = torch.exp(s - want_lse[:, None])
            want, a = p @ v, p @ v.abs()
            f = p.max(-1).values[:, None] * v.abs().sum(0)
            err = (o[r:r + 64, h].double() - want).abs()
            bound = 2.0 ** -8 * want.abs() + (step + 2.0 ** -12 + 2 * score_error) * a + (2.0 ** -32 * f if e4m3 else 0.0)
            assert bool((err <= bound).all()), f"head {h}: O off by {float((err / bound).max()):.2f} times the bound"
            # taken together: the output's roundings and the weights' are independent
            rms = err.square().mean().sqrt() / a.square().mean().sqrt()
            assert float(rms) <= 2.0 ** -8 + score_error, f"head {h}: O off by {float(rms):.2e} rms"
            off = (lse[h, r:r + 64].double() - want_lse).abs().max()
            assert float(off) <= 6e-5 + score_error, f"head {h}: lse off by {float(off):.2e}"


@pytest.mark.parametrize("hint", [1, 20, 400])  # 16 columns, 32 columns, tiles
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n_seq,keys,D,gap", [
    (1, 8192, 128, 12.0), (1, 32768, 128, 12.0), (296, 8192, 128, 10.0), (296, 8192, 128, 13.0), (296, 32768, 128, 11.0),
    (296, 32768, 128, 12.0), (296, 32768, 128, 14.0), (296, 32001, 64, 12.0)])
def test_one_key_far_above(n_seq, keys, D, gap, e4m3, hint):
    # 296 sequences are two whole units for each of 148 CTAs; one sequence is cut into pieces
    _check(n_seq, keys, 1, 1, D, gap, e4m3, hint)


@pytest.mark.parametrize("hint", [4, 8, 400])  # 16 and 32 columns of real rows, tiles
def test_one_key_far_above_grouped_drafts(hint):
    _check(40, 20000, 8, 2, 128, 12.0, True, hint, new=4)


@pytest.mark.parametrize("hint", [1, 20, 400])
def test_one_key_far_above_a_million(hint):
    # 18.5 nats: each other weight is near 2^-27 of the largest, all together 1 % of the row
    _check(148, 1 << 20, 1, 1, 64, 18.5, True, hint)


@pytest.mark.parametrize("hint", [1, 20, 400])
@pytest.mark.parametrize("n_seq,keys", [(1, 700), (1, 20000), (300, 20000)])
@pytest.mark.parametrize("v_scale", [2.0 ** -124, 2.0 ** 110])
def test_value_scales_at_the_ends(hint, n_seq, keys, v_scale):
    """A power of two as v_scale changes the output's exponent and nothing else (sums, factors and pieces in 32 bits
    have room for it; an output above 2^-126 is a normal number)."""
    q, cache = _batch(n_seq, keys, 2, 1, 128, 0.0, True)
    unit = _attn().PagedKV(cache.k, cache.v, cache.page_table, cache.seq_len, cache.q_start, k_scale=cache.k_scale)
    scaled = _attn().PagedKV(cache.k, cache.v, cache.page_table, cache.seq_len, cache.q_start, k_scale=cache.k_scale,
                             v_scale=v_scale)
    o1, lse1 = _attn().fwd_paged(unit, q, causal=False, max_new=hint)
    o2, lse2 = _attn().fwd_paged(scaled, q, causal=False, max_new=hint)
    assert _attn().device_status() == 0
    assert torch.equal(lse1, lse2)
    want = o1.double() * v_scale
    normal = (want.abs() >= 2.0 ** -125) & (o1 != 0)
    # (what is checked: at 2^-124 all but outputs below 1/2; they are near 25 N(0, 1), each channel's mean as stored: 1.6 %)
    assert float(normal.float().mean()) > 0.95
    # the pieces' fp32 rows lose nothing above 2^-126 either: what is left is one bf16 step where a piece's part is below it
    off = (o2.double() - want).abs()
    assert bool((off[normal] <= 2.0 ** -7 * want[normal].abs()).all())
    assert float((off[normal] != 0).float().mean()) < 0.01
