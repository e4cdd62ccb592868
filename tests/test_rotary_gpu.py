"""Rotary positions (attn_rope) against the fp64 oracle, and in the training step.

Tolerance: fp32 products and one rounding to bf16: half a step (2^-8 relative to the value) and
2^-21 of the pair's length for the fp32 arithmetic (cos and sin within 2^-23, two products and a sum)."""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from oracle import reference as ref
from tests import parity

pytestmark = pytest.mark.gpu


def _attn():
    import attention_attn_fwd_10_b200 as attn

    return attn


def _freq(n, base=10000.0):
    return (base ** (-torch.arange(n, dtype=torch.float64) / n)).float()


def _check(y, want, what=""):
    y = parity.to_np(y)
    err = np.abs(y - want)
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * np.abs(want).max() + 1e-38
    assert np.all(err <= bound), f"{what}: {err.max():.3e}"


@pytest.mark.parametrize("D,n_freq", [(64, 32), (128, 64), (128, 32), (128, 12), (64, 4), (64, 20), (128, 40)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,H_q,H_k", [(1, 1, 1), (7, 3, 1), (300, 32, 8), (33, 200, 0)])
def test_shapes(D, n_freq, interleaved, tokens, H_q, H_k):
    g = torch.Generator().manual_seed(tokens + n_freq)
    q = torch.randn((tokens, H_q, D), generator=g).bfloat16()
    k = torch.randn((tokens, H_k, D), generator=g).bfloat16() if H_k else None
    pos = torch.randint(-5000, 5000, (tokens,), generator=g, dtype=torch.int32)
    freq = _freq(n_freq)
    r = _attn().Rotary(freq.cuda(), interleaved=interleaved)
    for inverse in (False, True):
        got = _attn().rope(q.cuda(), None if k is None else k.cuda(), rotary=r, positions=pos.cuda(), inverse=inverse)
        for x, y in zip((q, k), got if H_k else (got,)):
            _check(y, oracle.rotate(x, pos.numpy()[None], freq, interleaved=interleaved, inverse=inverse))
            # the dims that do not turn are passed on as they are
            assert torch.equal(y.cpu()[..., 2 * n_freq:], x[..., 2 * n_freq:])


@pytest.mark.parametrize("sections", [(16, 24, 24), (0, 64), (64, 0), (1, 2, 3, 58), (13, 0, 51)])
def test_axes(sections):
    g = torch.Generator().manual_seed(3)
    q = torch.randn((2, 37, 4, 128), generator=g).bfloat16()
    pos = torch.randint(0, 4000, (len(sections), 2, 37), generator=g, dtype=torch.int32)
    freq = _freq(64)
    y = _attn().rope(q.cuda(), rotary=_attn().Rotary(freq.cuda(), sections=sections), positions=pos.cuda())
    want = oracle.rotate(q.flatten(0, 1), pos.flatten(1).numpy(), freq, sections)
    _check(y.flatten(0, 1), want)


@pytest.mark.parametrize("pos", [0, 1, -1, 1_000_003, 2 ** 31 - 1, -2 ** 31])
def test_far_positions(pos):
    # exact angles: an fp32 product would be off by whole turns' fractions here
    q = torch.randn((1, 2, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    freq = _freq(64)
    p = torch.tensor([pos], dtype=torch.int32)
    y = _attn().rope(q.cuda(), rotary=_attn().Rotary(freq.cuda()), positions=p.cuda())
    _check(y, oracle.rotate(q, p.numpy()[None], freq))


def test_default_positions_restart_in_each_row():
    q = torch.randn((3, 50, 2, 64), generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    r = _attn().Rotary(_freq(32).cuda())
    p = torch.arange(50, dtype=torch.int32, device="cuda").expand(3, 50).contiguous()
    assert torch.equal(_attn().rope(q, rotary=r), _attn().rope(q, rotary=r, positions=p))


def test_strides_in_place_streams_and_graph():
    attn = _attn()
    qkv = torch.randn((41, 8 + 2 + 2, 128), generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    q, k = qkv[:, :8], qkv[:, 8:10]  # slices of a fused projection
    r = attn.Rotary(_freq(64).cuda())
    want = attn.rope(q.contiguous(), k.contiguous(), rotary=r)
    got = attn.rope(q, k, rotary=r)
    assert got[0].is_contiguous() and all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = attn.rope(q, k, rotary=r, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    v = qkv[:, 10:].clone()
    graph = torch.cuda.CUDAGraph()
    scratch = qkv.clone()
    with torch.cuda.graph(graph):
        attn.rope(scratch[:, :8], scratch[:, 8:10], rotary=r, q_out=scratch[:, :8], k_out=scratch[:, 8:10])
    scratch.copy_(qkv)
    graph.replay()
    assert torch.equal(scratch[:, :8], want[0]) and torch.equal(scratch[:, 8:10], want[1])
    assert torch.equal(scratch[:, 10:], v)


def test_empty():
    attn = _attn()
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert attn.rope(q, rotary=attn.Rotary(_freq(32).cuda())).shape == q.shape


def test_refusals():
    attn = _attn()
    freq = _freq(32).cuda()
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(rotary=attn.Rotary(freq, sections=(8, 24))),  # several axes without positions
                dict(rotary=attn.Rotary(freq), positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(rotary=attn.Rotary(freq), positions=torch.zeros(4, dtype=torch.int64, device="cuda")),
                dict(rotary=attn.Rotary(freq), positions=torch.zeros(4, dtype=torch.int32)),
                dict(rotary=attn.Rotary(freq), k=torch.zeros((5, 2, 64), dtype=torch.bfloat16, device="cuda")),
                dict(rotary=attn.Rotary(freq), q_out=torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            attn.rope(q, **bad)
    with pytest.raises(TypeError):
        attn.rope(q.float(), rotary=attn.Rotary(freq))
    with pytest.raises(ValueError):
        attn.rope(q.transpose(0, 1), rotary=attn.Rotary(freq))  # heads that are not dense
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        attn.rope(q, rotary=attn.Rotary(freq[:6]))  # not a multiple of 4
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        attn.rope(q, rotary=attn.Rotary(_freq(64).cuda()))  # more than the head has
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        attn.rope(q, q[:1].expand(4, 2, 64), rotary=attn.Rotary(freq))  # tokens that share a place


def _loss(q, k, v, do, pos, freq, scale):
    """sum(do * attention(rotated q, rotated k, v)) in fp64, causal."""
    B, S = q.shape[:2]
    qr = oracle.rotate(q.reshape(B * S, *q.shape[2:]), pos, freq).reshape(q.shape)
    kr = oracle.rotate(k.reshape(B * S, *k.shape[2:]), pos, freq).reshape(k.shape)
    o, _ = ref.forward(qr, kr, v, True, scale)
    return float((o * do).sum()), qr, kr


@pytest.mark.parametrize("pipeline", [False, True])
def test_training_step_gradients(pipeline):
    """fwd_bwd(rotary=) and FwdBwdPipeline(rotary=): dq, dk are the gradients of the unrotated q, k: against
    the analytic formula and against central differences of the fp64 loss."""
    attn = _attn()
    B, S, H, D = 1, 130, 2, 64
    g = torch.Generator().manual_seed(11)
    q, k, v, do = (torch.randn((B, S, H, D), generator=g).bfloat16() for _ in range(4))
    freq, scale = _freq(32), D ** -0.5
    rotary = attn.Rotary(freq.cuda())
    if pipeline:
        pinned = [t.pin_memory() for t in (q, k, v, do)]
        out = {n: torch.empty((B, S, H, D), dtype=torch.bfloat16).pin_memory() for n in ("o", "dq", "dk", "dv")}
        out["lse"] = torch.empty((B, H, S)).pin_memory()
        pipe = attn.FwdBwdPipeline(B, S, S, H, H, D, causal=True, rotary=rotary)
        for _ in range(3):
            pipe.submit(*pinned, out)
        pipe.synchronize()
    else:
        out = attn.fwd_bwd(q, k, v, do, causal=True, rotary=rotary)
    assert attn.device_status() == 0
    pos = np.arange(S)[None]
    q64, k64, v64, do64 = (ref.to_f64(t) for t in (q, k, v, do))
    _, qr, kr = _loss(q64, k64, v64, do64, pos, freq, scale)
    o_ref, _ = ref.forward(qr, kr, v64, True, scale)
    # the rotated q and k are rounded to bf16 before the forward: scores off by 2^-7 at most relative
    # to |q||k| scale, beside the forward's own tolerance
    parity.check_o(out["o"], o_ref, "o", v_absmax=float(np.abs(v64).max()))
    dqr, dkr, dv = ref.backward(qr, kr, v64, do64, True, scale)
    dq = oracle.rotate(dqr[0], pos, freq, inverse=True)[None]
    dk = oracle.rotate(dkr[0], pos, freq, inverse=True)[None]
    for name, want in (("dq", dq), ("dk", dk), ("dv", dv)):
        parity.check_grad(out[name], want, name)
    rng = np.random.default_rng(0)
    for name, x in (("dq", q64), ("dk", k64)):
        d = rng.standard_normal(x.shape)
        h = 1e-5
        args = {"dq": q64, "dk": k64}
        vals = []
        for sgn in (1, -1):
            a = dict(args)
            a[name] = x + sgn * h * d
            vals.append(_loss(a["dq"], a["dk"], v64, do64, pos, freq, scale)[0])
        slope = (vals[0] - vals[1]) / (2 * h)
        got = float((parity.to_np(out[name]) * d).sum())
        # each element within 3e-2 of the largest gradient (check_grad), summed over independent directions
        assert abs(got - slope) <= 3e-2 * np.abs(want).max() * np.sqrt(x.size), (name, got, slope)


def test_training_step_on_another_stream():
    attn = _attn()
    g = torch.Generator().manual_seed(12)
    q, k, v, do = (torch.randn((2, 200, 2, 64), generator=g).bfloat16() for _ in range(4))
    r = attn.Rotary(_freq(32).cuda())
    torch.cuda.synchronize()
    a = attn.fwd_bwd(q, k, v, do, causal=True, rotary=r)
    b = attn.fwd_bwd(q, k, v, do, causal=True, rotary=r, stream=torch.cuda.Stream())
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["dk"], b["dk"]) and torch.equal(a["dv"], b["dv"])


def test_training_step_needs_equal_lengths():
    attn = _attn()
    q, k = torch.zeros((1, 4, 1, 64)).bfloat16(), torch.zeros((1, 5, 1, 64)).bfloat16()
    r = attn.Rotary(_freq(32).cuda())
    with pytest.raises(ValueError, match="S_q == S_k"):
        attn.fwd_bwd(q, k, k, q, rotary=r)
    with pytest.raises(ValueError, match="S_q == S_k"):
        attn.FwdBwdPipeline(1, 4, 5, 1, 1, 64, rotary=r)


@pytest.mark.parametrize("H_q,H_kv", [(2, 2), (4, 1)])
@pytest.mark.parametrize("pipeline", [False, True])
def test_training_step_gradients_along_themselves(pipeline, H_q, H_kv):
    """dq and dk against the formula's as a whole, and against the fp64 loss's slope along the formula's: that
    direction's slope is the gradient's squared norm, so a gradient that is missing, negated or left unrotated shows.

    Tolerance, relative to the gradient's norm: rounding to bf16 is at most 2^-8 of a value, 2^-8 / sqrt(3) rms.  q' and
    k': a score (rms 1) is off by sqrt(2) times that; P's rounding, dS's, k' (q') in the product, and the gradient's two
    (before and after it is turned back): sqrt(2 + 1 + 1 + 1 + 2) 2^-8 / sqrt(3) = 6e-3 in all; 2^-6 holds it 2.6 times."""
    attn = _attn()
    B, S, D = 2, 130, 64
    g = torch.Generator().manual_seed(13)
    q, do = (torch.randn((B, S, H_q, D), generator=g).bfloat16() for _ in range(2))
    k, v = (torch.randn((B, S, H_kv, D), generator=g).bfloat16() for _ in range(2))
    where = torch.randint(0, 5000, (B, S), generator=g, dtype=torch.int32)
    freq, scale = _freq(32), D ** -0.5
    rotary = attn.Rotary(freq.cuda())
    if pipeline:
        out = {n: torch.empty_like(t).pin_memory() for n, t in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
        out["lse"] = torch.empty((B, H_q, S)).pin_memory()
        pipe = attn.FwdBwdPipeline(B, S, S, H_q, H_kv, D, causal=True, rotary=rotary, positions=where.cuda())
        pipe.submit(*(t.pin_memory() for t in (q, k, v, do)), out)
        pipe.synchronize()
    else:
        out = attn.fwd_bwd(q, k, v, do, causal=True, rotary=rotary, positions=where)
    assert attn.device_status() == 0
    pos = where.reshape(1, -1).numpy()
    q64, k64, v64, do64 = (ref.to_f64(t) for t in (q, k, v, do))

    def turn(x, inverse=False):
        return oracle.rotate(x.reshape(B * S, *x.shape[2:]), pos, freq, inverse=inverse).reshape(x.shape)

    dqr, dkr, dv = ref.backward(turn(q64), turn(k64), v64, do64, True, scale)
    want = {"dq": turn(dqr, inverse=True), "dk": turn(dkr, inverse=True), "dv": dv}
    for name, w in want.items():
        got = parity.to_np(out[name])
        assert np.linalg.norm(got - w) <= 2.0 ** -6 * np.linalg.norm(w), name
    for name in ("dq", "dk"):
        w, h = want[name], 1e-5
        loss = []
        for sgn in (1, -1):
            at = {"dq": q64, "dk": k64}
            at[name] = at[name] + sgn * h * w
            loss.append(_loss(at["dq"], at["dk"], v64, do64, pos, freq, scale)[0])
        slope = (loss[0] - loss[1]) / (2 * h)
        assert abs(float((w * w).sum()) - slope) <= 1e-5 * slope, name  # the formula itself
        assert abs(float((parity.to_np(out[name]) * w).sum()) - slope) <= 2.0 ** -6 * slope, name


@pytest.mark.parametrize("shape", [(64,), (4, 64), (4, 1, 64), ()])
@pytest.mark.parametrize("rotary", [False, True])
def test_training_step_refuses_other_shapes(shape, rotary):
    attn = _attn()
    x = torch.zeros(shape).bfloat16()
    with pytest.raises(ValueError, match="4-D"):
        attn.fwd_bwd(x, x, x, x, rotary=attn.Rotary(_freq(32).cuda()) if rotary else None)
