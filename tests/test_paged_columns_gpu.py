"""Paged attention with few rows as MMA columns, 16 and 32 of them: many units per CTA (their pieces follow one
another through the same rings), small and odd pages, maxima that move in every block, calls at once and replayed."""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from tests.paged_cases import check_attend, handle, make, to_gpu

pytestmark = pytest.mark.gpu


def _attn():
    import attention_attn_fwd_10_b200 as attn

    return attn


def _check(x, hint, e4m3, causal=True, score_error=0.0):
    g = to_gpu(x)
    scale = x["q"].shape[2] ** -0.5
    o, lse = _attn().fwd_paged(handle(_attn(), g), g["q"], causal=causal, max_new=hint)
    torch.cuda.synchronize()
    assert _attn().device_status() == 0
    o_ref, lse_ref, a, f = oracle.attend(x["q"], x["k_cache"], x["v_cache"], x["page_table"].numpy(), x["keys"], x["start"],
                                         causal, scale, x["k_scale"], x["v_scale"])
    # fp16 weights over an e4m3 cache: no allowance for a floor under them (2^-32 of the largest, some hundred keys)
    check_attend(o, lse, (o_ref, lse_ref, a, 0 * f), np.arange(x["start"][0], x["start"][-1]), e4m3=e4m3,
                 score_error=score_error)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("group,most", [(4, 4), (4, 8), (8, 4), (16, 1), (31, 1)])
def test_many_units_per_cta(e4m3, D, page, group, most):
    rng = np.random.default_rng(group * most + page)
    B = 330  # times two kv heads: four or five units a CTA
    new = [int(n) for n in rng.integers(0, most + 1, B)]
    keys = [int(k) for k in rng.choice([0, 1, 5, 127, 128, 129, 255, 256, 257, 300, 511, 700], B)]
    x = make(new, keys, 2 * group, 2, D, page, e4m3=e4m3, seed=B + page)
    _check(x, most, e4m3, causal=bool(most > 1))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hint", [1, 20, 400])
@pytest.mark.parametrize("step", [3.0, 12.0, 40.0])
def test_maxima_that_move_in_every_block(e4m3, D, hint, step):
    """Scores that rise by `step` nats from one 128-key block to the next (12 nats are 17 binary places: every
    block rescales), so that the last keys decide, and fall again in the second sequence."""
    x = make([1, 1], [700, 1000], 1, 1, D, 64, e4m3=e4m3, seed=3)
    x["q"][..., 0] = 4.0
    for b, n in enumerate(x["keys"]):
        for j in range(n):
            level = (j if b == 0 else n - 1 - j) // 128
            k = min(step * level * D ** 0.5 / 4.0 / x["k_scale"], 448.0 if e4m3 else 1e4)
            x["k_cache"][int(x["page_table"][b, j // 64]), j % 64, 0, 0] = torch.tensor(k).to(x["k_cache"].dtype)
    top = float(max((x["q"].float() @ x["k_cache"][x["page_table"][b, : -(-n // 64)].long()].float().nan_to_num()
                     .flatten(0, 1)[:n, 0].T).abs().max() for b, n in enumerate(x["keys"]))) * x["k_scale"] * D ** -0.5
    # the fp32 sums of D products, the largest score and some 10 more of other signs
    _check(x, hint, e4m3, causal=False, score_error=D * 2.0 ** -24 * (top + 10))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [4, 8])
def test_at_once_and_replayed(D, new):
    """e4m3, 16 and 32 columns: several streams at once, and a captured call whose lengths change between replays."""
    attn = _attn()
    B = 70
    x = make([new] * B, [150 + 37 * b for b in range(B)], 8, 2, D, 64, e4m3=True, seed=6)
    g = to_gpu(x)
    cache = handle(attn, g)
    first = attn.fwd_paged(cache, g["q"], max_new=new)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    more = [attn.fwd_paged(cache, g["q"], max_new=new, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first[0]) and torch.equal(lse, first[1]) for o, lse in more)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = attn.fwd_paged(cache, g["q"], max_new=new)
    lens = g["seq_len"].clone()
    for cut in (0, 61, 149 - new, 0):
        g["seq_len"].copy_(lens - cut)
        want = attn.fwd_paged(cache, g["q"], max_new=new)
        o.fill_(7.0)
        graph.replay()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(o, first[0]) and attn.device_status() == 0
