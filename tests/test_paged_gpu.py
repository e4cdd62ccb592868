"""The paged cache: append (attn_paged_append) and attention (attn_fwd_paged) against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from oracle import reference as ref
from tests import parity
from tests.paged_cases import E4M3, check_attend, handle, make, to_cache, to_gpu

pytestmark = pytest.mark.gpu


def _attn():
    import attention_attn_fwd_10_b200 as attn

    return attn


def _freq(n):
    return (10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).float()


def _attend(x, causal=True, scale=None, **kw):
    g = to_gpu(x)
    D = x["q"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    o, lse = _attn().fwd_paged(handle(_attn(), g), g["q"], causal=causal, scale=scale, **kw)
    torch.cuda.synchronize()
    assert _attn().device_status() == 0
    want = oracle.attend(x["q"], x["k_cache"], x["v_cache"], x["page_table"].numpy(), x["keys"], x["start"], causal, scale,
                         x["k_scale"], x["v_scale"])
    return o, lse, want


def _rows(x):
    return np.arange(x["start"][0], x["start"][-1])


# ------------------------------------------------------------------------------------------- append

def _append_want(x, k, v, q, pos, freq, sections, interleaved, e4m3):
    T = k.shape[0]
    key = np.zeros(T, dtype=np.int64)
    where = oracle.slots(x["page_table"].numpy(), x["keys"], x["start"], x["k_cache"].shape[1])
    for t, _, j, _, _ in where:
        key[t] = j
    p = key[None] if pos is None else pos.numpy()
    kr = oracle.rotate(k, p, freq, sections, interleaved)
    qr = oracle.rotate(q, p, freq, sections, interleaved)
    return where, kr, ref.to_f64(v), qr


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,page,H_q,H_kv,n_freq,axes,interleaved", [
    (128, 16, 8, 2, 64, 1, False), (64, 48, 3, 3, 32, 3, True), (128, 64, 5, 1, 12, 1, True), (64, 128, 16, 4, 16, 2, False)])
def test_append(e4m3, D, page, H_q, H_kv, n_freq, axes, interleaved):
    new, keys = [1, 0, 40, 3, 17], [1, 50, 40, 200, 65]
    x = make(new, keys, H_q, H_kv, D, page, e4m3=e4m3, seed=D + page, extra_rows=2, poison=False)
    T = x["q"].shape[0]
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((T, H_kv, D), generator=g).bfloat16() for _ in range(2))
    freq = _freq(n_freq)
    sections = None if axes == 1 else (n_freq - (axes - 1) * (n_freq // axes),) + (n_freq // axes,) * (axes - 1)
    pos = None if axes == 1 else torch.randint(0, 9000, (axes, T), generator=g, dtype=torch.int32)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    d = to_gpu(x)
    rotary = _attn().Rotary(freq.cuda(), sections=sections, interleaved=interleaved)
    q_out = torch.full_like(d["q"], 7.0)
    cache = handle(_attn(), d)
    got = _attn().paged_append(cache, k.cuda(), v.cuda(), q=d["q"], rotary=rotary,
                               positions=None if pos is None else pos.cuda(), q_out=q_out)
    assert got is q_out and _attn().device_status() == 0
    where, kr, vr, qr = _append_want(x, k, v, x["q"], pos, freq, sections, interleaved, e4m3)
    kc, vc = d["k_cache"].cpu(), d["v_cache"].cpu()
    written = torch.zeros(kc.shape[:2], dtype=torch.bool)
    step = 2.0 ** -4 if e4m3 else 2.0 ** -8  # half a step of the stored type, relative
    floor = 2.0 ** -10 if e4m3 else 0.0      # e4m3's smallest step, halved
    for t, _, _, page_i, slot in where:
        written[page_i, slot] = True
        for c, r, s in ((kc, kr, x["k_scale"]), (vc, vr, x["v_scale"])):
            want = np.clip(r[t] / s, -448, 448) if e4m3 else r[t]
            err = np.abs(ref.to_f64(c[page_i, slot].float()) - want)
            assert np.all(err <= step * np.abs(want) + floor + 2.0 ** -20 * np.abs(want).max())
    as_bits = torch.uint8 if e4m3 else torch.int16
    for c, old in ((kc, before[0]), (vc, before[1])):  # nothing else is touched
        assert torch.equal(c.view(as_bits)[~written], old.view(as_bits)[~written])
    rows = _rows(x)
    err = np.abs(parity.to_np(q_out)[rows] - qr[rows])
    assert np.all(err <= 2.0 ** -8 * np.abs(qr[rows]) + 2.0 ** -20 * np.abs(qr).max())
    assert torch.all(q_out[x["start"][-1]:] == 7.0)  # rows behind the last sequence


def test_append_without_rotation_and_strided_layouts():
    attn = _attn()
    x = make([3, 2], [20, 5], 4, 2, 64, 16, seed=2, poison=False)
    T, n_pages = 5, x["k_cache"].shape[0]
    qkv = torch.randn((T, 4 + 2 + 2, 64), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    d = to_gpu(x)
    plain = handle(attn, d)
    assert attn.paged_append(plain, k, v) is None
    # [n_pages, 2, H_kv, page, D]: k and v as slices of one pool, heads outside the slots
    pool = torch.zeros((n_pages, 2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    other = attn.PagedKV(pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2), d["page_table"], d["seq_len"], d["q_start"])
    attn.paged_append(other, k, v)
    for t, _, _, page, slot in oracle.slots(x["page_table"].numpy(), x["keys"], x["start"], 16):
        assert torch.equal(d["k_cache"][page, slot], k[t]) and torch.equal(d["v_cache"][page, slot], v[t])
        assert torch.equal(pool[page, 0, :, slot], k[t]) and torch.equal(pool[page, 1, :, slot], v[t])
    # the same with rotation, q in place in its own buffer
    r = attn.Rotary(_freq(32).cuda())
    want = attn.paged_append(plain, k, v, q=q, rotary=r)
    mine = q.contiguous()
    assert attn.paged_append(other, k, v, q=mine, rotary=r, q_out=mine) is mine
    assert torch.equal(mine, want)
    for t, _, _, page, slot in oracle.slots(x["page_table"].numpy(), x["keys"], x["start"], 16):
        assert torch.equal(pool[page, 0, :, slot], d["k_cache"][page, slot])
    assert attn.device_status() == 0


def test_append_saturates_and_keeps_nan():
    attn = _attn()
    x = make([1], [1], 1, 1, 64, 16, e4m3=True, poison=False)
    x["k_scale"], x["v_scale"] = 0.001, 1.0
    d = to_gpu(x)
    k = torch.full((1, 1, 64), 30.0).bfloat16().cuda()
    v = torch.tensor([float("inf"), float("-inf"), float("nan"), 1.0] * 16).bfloat16().view(1, 1, 64).cuda()
    attn.paged_append(handle(attn, d), k, v)
    page = int(x["page_table"][0, 0])
    assert torch.all(d["k_cache"][page, 0].float() == 448)
    got = d["v_cache"][page, 0, 0].float().cpu()
    assert torch.equal(got[:2], torch.tensor([448.0, -448.0])) and torch.isnan(got[2]) and got[3] == 1


# ------------------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,keys", [
    ([1], [1]), ([1], [127]), ([1], [128]), ([1], [129]), ([1], [2000]),
    ([1, 1, 1, 1, 1], [5, 300, 1, 1024, 640]),
    ([4, 4, 2], [4, 333, 1000]),
    ([130], [130]), ([257], [700]), ([64, 1, 0, 200, 1], [64, 513, 77, 900, 1])])
def test_attend_lengths(e4m3, D, new, keys):
    x = make(new, keys, 8, 2, D, 16, e4m3=e4m3, seed=sum(keys) + D)
    for causal in (True, False):
        o, lse, want = _attend(x, causal, max_new=max(new))
        check_attend(o, lse, want, _rows(x), f"causal={causal}", e4m3=e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (4, 4), (3, 1), (10, 2), (14, 2), (16, 1), (17, 1), (32, 1), (33, 1), (71, 1),
                                      (128, 1), (128, 2)])
@pytest.mark.parametrize("new,keys", [([1, 1], [300, 150]), ([3, 1, 5], [77, 260, 6])])
def test_attend_heads(e4m3, H_q, H_kv, new, keys):
    x = make(new, keys, H_q, H_kv, 128, 32, e4m3=e4m3, seed=H_q)
    o, lse, want = _attend(x, max_new=max(new))
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 48, 64, 80, 112, 128, 144, 256, 1024])
def test_attend_pages(e4m3, page):
    x = make([1, 150, 2], [500, 300, 1030], 4, 2, 128, page, e4m3=e4m3, seed=page)
    o, lse, want = _attend(x)
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))


@pytest.mark.parametrize("hint", [0, 1, 3, 8, 1000000])
def test_attend_any_hint(hint):
    # the hint chooses the kernel; more new tokens than it says are served all the same
    x = make([3, 1, 70, 300], [900, 128, 70, 513], 8, 2, 128, 64, seed=hint % 97)
    o, lse, want = _attend(x, max_new=hint)
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))


@pytest.mark.parametrize("hint", [1, 400])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_rows_without_keys(hint, e4m3):
    # no keys at all; more new tokens than keys (the first see none)
    x = make([2, 300, 1, 40], [0, 100, 1, 7], 4, 1, 128, 16, e4m3=e4m3, seed=4)
    o, lse, want = _attend(x, max_new=hint)
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))
    assert torch.all(o[:2] == 0) and torch.all(torch.isneginf(lse[:, :2]))
    assert torch.all(o[2:202] == 0) and torch.all(torch.isneginf(lse[:, 2:202]))


@pytest.mark.parametrize("hint", [1, 400])
def test_attend_leaves_other_rows(hint):
    # rows before the first sequence and behind the last one keep what they held
    x = make([2, 30], [200, 300], 4, 2, 128, 16, seed=5, extra_rows=9)
    x["start"] = [s + 3 for s in x["start"]]
    x["q_start"] = x["q_start"] + 3
    out = torch.full(x["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, x["q"].shape[0]), 7.0, device="cuda")
    o, lse, want = _attend(x, out=out, lse=lse, max_new=hint)
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))
    rest = np.setdiff1d(np.arange(x["q"].shape[0]), _rows(x))
    assert torch.all(o[rest] == 7) and torch.all(lse[:, rest] == 7)


@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_many_sequences(e4m3):
    rng = np.random.default_rng(6)
    B = 300
    new = [int(n) for n in rng.choice([0, 1, 1, 1, 2, 9], B)]
    keys = [max(n, int(rng.integers(0, 400))) for n in new]
    x = make(new, keys, 4, 2, 64, 16, e4m3=e4m3, seed=6)
    o, lse, want = _attend(x)
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,keys", [([1], [33000]), ([5], [20011]), ([200], [9001])])
def test_attend_long(e4m3, new, keys):
    # one sequence split over every SM
    x = make(new, keys, 4, 1, 128, 64, e4m3=e4m3, seed=7)
    o, lse, want = _attend(x, max_new=max(new))
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))


@pytest.mark.parametrize("hint", [1, 400])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_extreme_scores(hint, e4m3):
    """Rows whose largest score comes late and is far above the rest (the running maximum moves), and queries
    of very different sizes, in every row's own scale."""
    x = make([2, 140], [900, 700], 4, 2, 128, 16, e4m3=e4m3, seed=8)
    q = x["q"].float()
    gain = torch.tensor([2.0 ** -20, 1.0, 0.25, 3.0])
    x["q"] = (q * gain[None, :, None]).bfloat16()
    # a key that matches the queries of head 0's group strongly, near each sequence's end and in its middle
    for b, n in enumerate(x["keys"]):
        for j in (n // 2, n - 1):
            page, slot = int(x["page_table"][b, j // 16]), j % 16
            big = 4.0 * q[x["start"][b], 1].float() / x["k_scale"]
            x["k_cache"][page, slot, 0] = big.clamp(-448, 448).to(x["k_cache"].dtype)
    o, lse, want = _attend(x, max_new=hint)
    # scores up to 51 here, sums of 128 products of one sign: 128 x 2^-24 x 51 = 3.9e-4
    check_attend(o, lse, want, _rows(x), e4m3=e4m3, score_error=3.9e-4)


def test_attend_shared_pages_and_strided_layouts():
    attn = _attn()
    x = make([1, 1], [70, 70], 4, 2, 64, 16, seed=9)
    # both sequences read the same pages (a common prefix, and here all of it)
    x["page_table"][1] = x["page_table"][0]
    o, lse, want = _attend(x)
    check_attend(o, lse, want, _rows(x), e4m3=bool(x["k_scale"] != 1.0))
    d = to_gpu(x)
    n = x["k_cache"].shape[0]
    pool = torch.empty((n, 2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    pool[:, 0].copy_(d["k_cache"].transpose(1, 2))
    pool[:, 1].copy_(d["v_cache"].transpose(1, 2))
    wide = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, : d["page_table"].shape[1]] = d["page_table"]
    other = attn.PagedKV(pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2), wide[:, :30], d["seq_len"], d["q_start"])
    fused = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    fused[:, :4] = d["q"]
    o2, lse2 = attn.fwd_paged(other, fused[:, :4], scale=0.125)
    check_attend(o2, lse2, want, _rows(x))
    assert attn.device_status() == 0


@pytest.mark.parametrize("hint", [1, 400])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_same_every_time_and_on_other_streams(hint, e4m3):
    attn = _attn()
    x = make([1, 60, 1], [4000, 600, 100], 8, 2, 128, 64, e4m3=e4m3, seed=10)
    d = to_gpu(x)
    cache = handle(attn, d)
    first = attn.fwd_paged(cache, d["q"], max_new=hint)
    again = attn.fwd_paged(cache, d["q"], max_new=hint)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    more = [attn.fwd_paged(cache, d["q"], max_new=hint, stream=s) for s in streams for _ in range(3)]  # at once
    torch.cuda.synchronize()
    for o, lse in [again, *more]:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    assert attn.device_status() == 0


@pytest.mark.parametrize("hint", [1, 400])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_many_ragged_chunks(hint, e4m3):
    """Chunks and single tokens, more units than CTAs, lengths around the 128-key blocks."""
    rng = np.random.default_rng(21)
    new = [int(n) for n in rng.choice([1, 1, 2, 33, 64, 65, 127, 128, 129, 300], 40)]
    keys = [n + int(k) for n, k in zip(new, rng.choice([0, 1, 63, 127, 128, 200, 500], 40))]
    x = make(new, keys, 6, 2, 64, 48, e4m3=e4m3, seed=21)
    for causal in (True, False):
        o, lse, want = _attend(x, causal, max_new=hint)
        check_attend(o, lse, want, _rows(x), f"causal={causal}", e4m3=e4m3)


@pytest.mark.parametrize("hint", [1, 400])
def test_attend_whole_and_shared_stretches(hint):
    """Unit counts and lengths on both sides of the rules that lay the work out (short stretches of one piece,
    long ones that hold several units)."""
    for B, keys in ((1, 140), (1, 8000), (2, 2500), (7, 1111), (31, 515), (33, 515), (60, 1030)):
        x = make([1] * B, [keys + 13 * b for b in range(B)], 4, 2, 128, 64, seed=B, poison=False)
        o, lse, want = _attend(x, max_new=hint)
        check_attend(o, lse, want, _rows(x), f"{B} x {keys}")


def test_cache_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: pages at its far end."""
    attn = _attn()
    H_kv, D, page, n_pages = 8, 128, 128, 17000
    assert n_pages * page * H_kv * D > 2 ** 31
    x = make([3, 1], [300, 129], 16, H_kv, D, page, seed=22, poison=False)
    g = to_gpu(x)
    far = {}
    for name in ("k_cache", "v_cache"):
        far[name] = torch.empty((n_pages, page, H_kv, D), dtype=torch.bfloat16, device="cuda")
        far[name][-g[name].shape[0]:] = g[name]
    table = torch.where(g["page_table"] < 2 ** 29, g["page_table"] + n_pages - x["k_cache"].shape[0], g["page_table"])
    cache = attn.PagedKV(far["k_cache"], far["v_cache"], table.contiguous(), g["seq_len"], g["q_start"])
    o, lse = attn.fwd_paged(cache, g["q"])
    want = attn.fwd_paged(handle(attn, g), g["q"])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    k = torch.randn((4, H_kv, D), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    v = -k
    attn.paged_append(cache, k, v)
    for t, _, _, pg, slot in oracle.slots(table.cpu().numpy(), x["keys"], x["start"], page):
        assert pg > 16000
        assert torch.equal(far["k_cache"][pg, slot], k[t]) and torch.equal(far["v_cache"][pg, slot], v[t])
    assert attn.device_status() == 0


def test_calls_from_several_threads():
    import threading

    attn = _attn()
    xs = [make([1, 40], [700, 300 + 10 * i], 8, 2, 128, 16, e4m3=i % 2 == 1, seed=30 + i) for i in range(4)]
    gs = [to_gpu(x) for x in xs]
    want = [attn.fwd_paged(handle(attn, g), g["q"]) for g in gs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]

    def work(i):
        s = torch.cuda.Stream()
        cache = handle(attn, gs[i])
        for _ in range(20):
            got[i].append(attn.fwd_paged(cache, gs[i]["q"], stream=s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(4):
        assert len(got[i]) == 20
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    assert attn.device_status() == 0


@pytest.mark.skipif(not torch.cuda.is_available() or torch.cuda.device_count() < 2, reason="needs two devices")
def test_on_the_device_of_the_tensors():
    attn = _attn()
    x = make([1, 5], [300, 200], 4, 2, 128, 16, seed=40)
    want = oracle.attend(x["q"], x["k_cache"], x["v_cache"], x["page_table"].numpy(), x["keys"], x["start"], True, 128 ** -0.5)
    for d in (0, 1):
        g = {n: t.to(f"cuda:{d}") if isinstance(t, torch.Tensor) else t for n, t in x.items()}
        with torch.cuda.device(1 - d):  # the current device is another one
            o, lse = attn.fwd_paged(handle(attn, g), g["q"])
        torch.cuda.synchronize(d)
        assert o.device.index == d
        check_attend(o, lse, want, _rows(x), f"device {d}")


@pytest.mark.parametrize("hint", [1, 20, 400])
@pytest.mark.parametrize("e4m3", [False, True])
def test_waits_that_run_out_are_reported(hint, e4m3):
    """With a limit of 1 ns per wait the kernels give up, report it and leave; the next call is right again."""
    attn = _attn()
    x = make([1, 200, 1], [3000, 900, 700], 8, 4, 128, 16, e4m3=e4m3, seed=41)
    g = to_gpu(x)
    cache = handle(attn, g)
    want = attn.fwd_paged(cache, g["q"], max_new=hint)
    assert attn.device_status() == 0
    attn.set_wait_limit_ns(1)
    try:
        for _ in range(3):
            attn.fwd_paged(cache, g["q"], max_new=hint)
        status = attn.device_status()
    finally:
        attn.set_wait_limit_ns(0)
    assert status == 5
    o, lse = attn.fwd_paged(cache, g["q"], max_new=hint)
    assert attn.device_status() == 0
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_run(e4m3):
    """Prompts of two sequences in chunks, then single tokens, through append and attention, against causal
    attention of the whole sequences; the decoding steps are one captured graph whose lengths move on the device."""
    attn = _attn()
    H_q, H_kv, D, page, freq = 8, 2, 128, 16, _freq(64)
    total, prompt = [150, 97], [140, 90]
    g = torch.Generator().manual_seed(13)
    Q, K, V = ([torch.randn((n, h, D), generator=g).bfloat16() for n in total] for h in (H_q, H_kv, H_kv))
    k_scale, v_scale = (0.03125, 0.025) if e4m3 else (1.0, 1.0)
    dtype = E4M3 if e4m3 else torch.bfloat16
    k_cache, v_cache = (torch.zeros((24, page, H_kv, D), device="cuda").to(dtype) for _ in range(2))
    table = torch.randperm(24, generator=g)[:20].view(2, 10).int().cuda()
    seq_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    q_start = torch.zeros(3, dtype=torch.int32, device="cuda")
    cache = attn.PagedKV(k_cache, v_cache, table, seq_len, q_start, k_scale=k_scale, v_scale=v_scale)
    rotary = attn.Rotary(freq.cuda())
    scale = D ** -0.5
    done, outs = [0, 0], [[], []]

    def take(counts):
        rows = [t[b][done[b]:done[b] + c] for t in (Q, K, V) for b, c in enumerate(counts)]
        return [torch.cat(rows[2 * i:2 * i + 2]).cuda() for i in range(3)]

    for counts in ([100, 1], [40, 89]):
        q, k, v = take(counts)
        seq_len.copy_(torch.tensor([done[b] + counts[b] for b in range(2)], dtype=torch.int32))
        q_start.copy_(torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32))
        o, _ = attn.fwd_paged(cache, attn.paged_append(cache, k, v, q=q, rotary=rotary), scale=scale)
        for b, part in enumerate(o.split(counts)):
            outs[b].append(part)
            done[b] += counts[b]
    assert done == prompt
    # decoding: one graph for all steps; sequence 1 ends three steps before sequence 0
    q, k, v = (torch.zeros((2, h, D), dtype=torch.bfloat16, device="cuda") for h in (H_q, H_kv, H_kv))
    seq_len.copy_(torch.tensor([done[0] + 1, done[1] + 1], dtype=torch.int32))
    q_start.copy_(torch.tensor([0, 1, 2], dtype=torch.int32))
    keep = k_cache.clone(), v_cache.clone()
    o = torch.empty((2, H_q, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(attn.fwd_paged_workspace_size(H_q, H_kv, D), dtype=torch.uint8, device="cuda")

    def step():
        return attn.fwd_paged(cache, attn.paged_append(cache, k, v, q=q, rotary=rotary), scale=scale, out=o, workspace=ws,
                              max_new=1)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    k_cache.copy_(keep[0])
    v_cache.copy_(keep[1])
    while done[0] < total[0]:
        counts = [1, int(done[1] < total[1])]
        rows = take(counts)
        for dst, src in zip((q, k, v), rows):
            dst[: sum(counts)] = src
        seq_len.copy_(torch.tensor([done[b] + counts[b] for b in range(2)], dtype=torch.int32))
        q_start.copy_(torch.tensor([0, 1, 1 + counts[1]], dtype=torch.int32))
        graph.replay()
        for b, part in enumerate(o[: sum(counts)].clone().split(counts)):
            outs[b].append(part)
            done[b] += counts[b]
    assert done == total and attn.device_status() == 0
    for b in range(2):
        pos = np.arange(total[b])[None]
        # what the cache and the kernel hold: rotated rows, rounded once
        qr = torch.from_numpy(oracle.rotate(Q[b], pos, freq)).float().bfloat16()
        kr = to_cache(torch.from_numpy(oracle.rotate(K[b], pos, freq)).float(), k_scale, e4m3)
        vr = to_cache(V[b].float(), v_scale, e4m3)
        k64, v64 = ref.to_f64(kr.float()) * k_scale, ref.to_f64(vr.float()) * v_scale
        want, _ = ref.forward(qr[None], k64[None], v64[None], True, scale)
        a, _ = ref.forward(qr[None], k64[None], np.abs(v64)[None], True, scale)
        got = parity.to_np(torch.cat(outs[b]))
        # a rotated value next to a border may round the other way on the GPU: one step of one input
        # moves a score by 2^-7 (2^-3 for e4m3) of its share; the bound of check_attend with that added
        extra = (2.0 ** -4 if e4m3 else 2.0 ** -8) * a[0]
        assert np.all(np.abs(got - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -7 * a[0] + extra)


def test_two_graphs_share_a_workspace():
    attn = _attn()
    a = to_gpu(make([1, 1], [3000, 100], 8, 2, 128, 64, seed=14))
    b = to_gpu(make([50], [2000], 8, 2, 128, 64, seed=15))
    ws = torch.empty(attn.fwd_paged_workspace_size(8, 2, 128), dtype=torch.uint8, device="cuda")
    want, graphs, outs = [], [], []
    for d in (a, b):
        cache = handle(attn, d)
        want.append(attn.fwd_paged(cache, d["q"]))
        out = torch.empty_like(d["q"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.fwd_paged(cache, d["q"], out=out, workspace=ws)
        graphs.append(graph)
        outs.append(out)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i][0])


# ------------------------------------------------------------------------------------------- bad indices, refusals

@pytest.mark.parametrize("hint", [1, 400])
@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "range", "start"])
def test_bad_indices_are_reported(what, hint):
    """Entries that lead outside the cache or the token rows: no access out of range, the status says so, the
    other sequences are served."""
    attn = _attn()
    x = make([2, 2], [100, 60], 4, 2, 128, 16, seed=16)
    good = _attend(x, max_new=hint)
    d = to_gpu(x)
    if what == "page":
        d["page_table"][1, 2] = x["k_cache"].shape[0]
    elif what == "negative page":
        d["page_table"][1, 0] = -5
    elif what == "length":
        d["seq_len"][1] = 16 * x["page_table"].shape[1] + 1000000
        d["page_table"][1] = torch.arange(x["page_table"].shape[1], device="cuda") % 4
    elif what == "negative length":
        d["seq_len"][1] = -7
    elif what == "range":
        d["q_start"][2] = 1000000000
    else:
        d["q_start"][0] = -3
    o, lse = attn.fwd_paged(handle(attn, d), d["q"], scale=128 ** -0.5, max_new=hint)
    assert attn.device_status() == 7
    if what not in ("range", "start"):
        assert torch.equal(o[:2], good[0][:2]) and torch.equal(lse[:, :2], good[1][:, :2])
    k = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    before = d["k_cache"].clone().view(torch.int16)
    attn.paged_append(handle(attn, d), k, k)
    if what not in ("page", "negative page"):  # the appended keys do not lie on those pages
        assert attn.device_status() == 7
    else:
        attn.device_status()
    changed = (d["k_cache"].view(torch.int16) != before).any(-1).any(-1).sum()
    assert changed <= 4
    o, lse = attn.fwd_paged(handle(attn, to_gpu(x)), to_gpu(x)["q"], scale=128 ** -0.5, max_new=hint)
    assert torch.equal(o, good[0]) and attn.device_status() == 0


@pytest.mark.parametrize("starts", [[0, 4, 1000000], [0, 5, 3], [0, 4, 3, 4], [0, 4, -2], [0, 4, 4, 5], [0] * 300 + [4, 9]])
@pytest.mark.parametrize("op", ["append", "attend"])
def test_bad_ranges_without_rows_are_reported(op, starts):
    """Ranges that no token row belongs to: past the rows, running backwards, among many sequences."""
    attn = _attn()
    n = len(starts) - 1
    T, page = 4, 16
    kc, vc = (torch.zeros((8, page, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = (torch.arange(n * 2, dtype=torch.int32, device="cuda") % 8).view(n, 2)
    lens = torch.full((n,), 20, dtype=torch.int32, device="cuda")

    def call(s):
        start = torch.tensor(s, dtype=torch.int32, device="cuda")
        x = torch.ones((T, 1, 64), dtype=torch.bfloat16, device="cuda")
        cache = attn.PagedKV(kc, vc, table, lens, start)
        if op == "append":
            attn.paged_append(cache, x, x)
        else:
            attn.fwd_paged(cache, x, max_new=1)
        return attn.device_status()

    assert call(starts) == 7
    assert call([0] + [T] * n) == 0


def test_handles_follow_their_tensors_or_refuse():
    """The handle goes by what it was made of: changed in place it follows, a replacement is refused."""
    attn = _attn()
    x = make([1, 1], [100, 60], 4, 2, 128, 16, seed=18)
    g = to_gpu(x)
    cache = handle(attn, g)
    cache.seq_len -= 1  # in place
    o, _ = attn.fwd_paged(cache, g["q"])
    y = make([1, 1], [100, 60], 4, 2, 128, 16, seed=18)
    y["seq_len"] = y["seq_len"] - 1
    h = to_gpu(y)
    assert torch.equal(o, attn.fwd_paged(handle(attn, h), h["q"])[0])
    for name, value in (("seq_len", g["seq_len"] + 1), ("page_table", g["page_table"].clone()), ("k", g["k_cache"].clone()),
                        ("q_start", g["q_start"].clone()), ("v", g["v_cache"].clone()), ("k_scale", 2.0), ("H_kv", 1)):
        with pytest.raises(AttributeError, match=name):
            setattr(cache, name, value)
    r = attn.Rotary(_freq(64).cuda())
    for name, value in (("inv_freq", _freq(32).cuda()), ("sections", (32, 32)), ("interleaved", True)):
        with pytest.raises(AttributeError, match=name):
            setattr(r, name, value)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hint", [1, 20, 400])
def test_lengths_that_change_meanwhile(hint, e4m3):
    """Another stream rewrites lengths and ranges, each content valid, while calls run: nothing outside the outputs and
    the workspace is written, and a call on settled lengths is right again."""
    attn = _attn()
    rng = np.random.default_rng(5)
    B = 150
    new = [int(n) for n in rng.choice([1, 2, 9, 40], B)]
    x = make(new, [n + int(k) for n, k in zip(new, rng.integers(300, 900, B))], 4, 2, 64, 64, e4m3=e4m3, seed=31, poison=False)
    g = to_gpu(x)
    g["page_table"].clamp_(max=x["k_cache"].shape[0] - 1)
    T = sum(new)
    size = attn.fwd_paged_workspace_size(4, 2, 64)
    out = torch.full((T + 64, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4 * T + 128,), 7.0, device="cuda")
    ws = torch.full((size + 65536,), 7, dtype=torch.uint8, device="cuda")
    o, l, w = out[32:32 + T], lse[64:64 + 4 * T].view(4, T), ws[32768:32768 + size]
    cache = handle(attn, g)
    want = attn.fwd_paged(cache, g["q"], max_new=hint)
    lens, starts = g["seq_len"].clone(), g["q_start"].clone()
    other = torch.tensor(sorted(rng.integers(0, T + 1, B + 1).tolist()), dtype=torch.int32, device="cuda")
    short = torch.tensor(rng.integers(0, 300, B), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for i in range(400):
            g["seq_len"].copy_(short if i % 2 == 0 else lens)
            g["q_start"].copy_(other if i % 3 == 0 else starts)
    for _ in range(40):
        attn.fwd_paged(cache, g["q"], max_new=hint, out=o, lse=l, workspace=w)
    torch.cuda.synchronize()
    assert attn.device_status() in (0, 7)
    for t, a, b, v in ((out, 32, 32 + T, 7.0), (lse, 64, 64 + 4 * T, 7.0), (ws, 32768, 32768 + size, 7)):
        assert bool((t[:a] == v).all()) and bool((t[b:] == v).all())
    g["seq_len"].copy_(lens)
    g["q_start"].copy_(starts)
    again = attn.fwd_paged(cache, g["q"], max_new=hint, out=o, lse=l, workspace=w)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1]) and attn.device_status() == 0


@pytest.mark.parametrize("length", [-1, 33, 2 ** 31 - 1])
def test_bad_lengths_without_rows_are_reported(length):
    attn = _attn()
    kc, vc = (torch.zeros((8, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    start = torch.tensor([0, 4, 4], dtype=torch.int32, device="cuda")
    x = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    for n, want in ((length, 7), (32, 0), (0, 0)):
        cache = attn.PagedKV(kc, vc, table, torch.tensor([20, n], dtype=torch.int32, device="cuda"), start)
        attn.paged_append(cache, x, x)
        assert attn.device_status() == want
        attn.fwd_paged(cache, x)
        assert attn.device_status() == want


def test_refusals():
    attn = _attn()
    d = to_gpu(make([1], [40], 4, 2, 64, 16, seed=17))
    base = (d["k_cache"], d["v_cache"], d["page_table"], d["seq_len"], d["q_start"])

    def cache(i=None, t=None, **kw):
        a = list(base)
        if i is not None:
            a[i] = t
        return attn.PagedKV(*a, **kw)

    for i, t in ((0, base[0][:, :8]), (1, base[1].transpose(1, 2).contiguous().transpose(1, 2)), (2, base[2][0]),
                 (3, torch.zeros(2, dtype=torch.int32, device="cuda")), (4, base[4][:1]), (0, base[0].cpu()),
                 (2, base[2].cpu())):
        with pytest.raises(ValueError):
            cache(i, t)
    for i, t in ((0, base[0].float()), (0, base[0].to(E4M3)), (2, base[2].long()), (3, base[3].long()), (4, base[4].long())):
        with pytest.raises(TypeError):
            cache(i, t)
    c = cache()
    q = d["q"]
    for bad in (q[0], q.cpu(), q.expand(1, 4, 64)[:, :, :32]):
        with pytest.raises(ValueError):
            attn.fwd_paged(c, bad)
    with pytest.raises(TypeError):
        attn.fwd_paged(c, q.half())
    for kw in (dict(out=q.float()), dict(lse=torch.zeros((1, 4), device="cuda")),
               dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            attn.fwd_paged(c, q, **kw)
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(max_new=-1)):
        with pytest.raises(RuntimeError, match="INVALID_ARG"):
            attn.fwd_paged(c, q, **kw)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        attn.fwd_paged(c, q[:, :3].contiguous())  # 3 heads over 2
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        attn.fwd_paged(cache(k_scale=2.0), q)  # a bf16 cache has no scales
    odd = torch.zeros((4, 24, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        attn.fwd_paged(attn.PagedKV(odd, odd.clone(), *base[2:]), q)  # pages of 24 keys
    over = torch.zeros(100000, dtype=torch.bfloat16, device="cuda").as_strided((4, 16, 2, 64), (2048, 64, 128, 1))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        attn.fwd_paged(attn.PagedKV(over, over, *base[2:]), q)  # elements that share a place
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    r = attn.Rotary(_freq(32).cuda())
    for bad in (dict(q=q), dict(q=torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda"), rotary=r),
                dict(positions=torch.zeros(1, dtype=torch.int32, device="cuda")), dict(q_out=q, rotary=r)):
        with pytest.raises(ValueError):
            attn.paged_append(c, k, k, **bad)
    with pytest.raises(ValueError):
        attn.paged_append(c, k, torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda"))
    assert attn.device_status() == 0


@pytest.mark.parametrize("max_new", [1, 300])
def test_lse_keeps_32_bits(max_new):
    """Rows that few keys dominate: the row's sum is as exact as its largest weights.  Bounds: a score is D / 16 partial
    sums and one across them, each cut at 2^-23 of at most sum |q k| scale, twice for the sums inside one; the row's
    sum 25 roundings of 2^-24, ex2 2^-22; exponent, maximum and scale 2^-24 of the largest score each, the result twice."""
    D, scale = 64, 64 ** -0.5
    x = make([max_new, 1], [700, 900], 8, 2, D, 64, q_gain=3.0, seed=41)
    _, lse, want = _attend(x, False, max_new=max_new)
    most = 0.0
    for b in range(2):
        k = np.abs(oracle.gather(x["k_cache"], x["page_table"].numpy()[b], x["keys"][b]))  # [keys, H_kv, D]
        q = np.abs(x["q"][x["start"][b]:x["start"][b + 1]].double().numpy())
        for h in range(8):
            most = max(most, float((q[:, h] @ k[:, h // 4].T).max()) * scale)
    bound = 2 * (D / 16 + 1) * 2.0 ** -23 * most + 25 * 2.0 ** -24 + 2.0 ** -22 + 5 * 2.0 ** -24 * most
    err = np.abs(parity.to_np(lse) - want[1])
    assert err.max() <= bound, f"lse {err.max():.3e} > {bound:.3e}"
