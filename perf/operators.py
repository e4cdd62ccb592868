"""The paged serving operators and the rotary positions, as cases to measure.

Three operators:
  rope     rotary positions with one to three axes on q and k, forward or inverse (the inverse is
           its backward pass);
  append   the new tokens' keys rotated and written, with their values, into a paged cache (bf16 or
           e4m3 with scales), and their queries rotated;
  attend   attention of each sequence's new tokens over its paged cache (output and logsumexp).

``run`` computes them in plain torch operations, or with the package's kernels where ``own`` is
true; ``exact`` states them in 64 bits.  Lengths follow from the case alone, values from the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------
# cases

def _rope(name, B, S, H_q, H_kv, D, axes=1, inverse=False, interleaved=False, start=0, rotated=None):
    return {"name": name, "op": "rope", "B": B, "S": S, "H_q": H_q, "H_kv": H_kv, "D": D, "axes": axes,
            "inverse": inverse, "interleaved": interleaved, "start": start, "rotated": rotated or D}


def _paged(name, op, B, new, ctx, H_q, H_kv, D, page, e4m3=False, single=0.0, ragged=True, axes=1,
           interleaved=False, causal=True):
    """B sequences of at most ``ctx`` keys, each with up to ``new`` new tokens (``single``: the
    share of the sequences that bring one token only)."""
    case = {"name": name, "op": op, "B": B, "new": new, "ctx": ctx, "H_q": H_q, "H_kv": H_kv, "D": D, "page": page,
            "e4m3": e4m3, "single": single, "ragged": ragged}
    if op == "append":
        return case | {"axes": axes, "interleaved": interleaved}
    return case | {"causal": causal}


def listed():
    return [
        # a short sequence: launch latency
        _rope("rope_short", 1, 256, 2, 2, 64),
        # the training step's q and k
        _rope("rope_train_8k", 2, 8192, 16, 16, 128),
        # the gradients of q and k of a video clip's tokens (time, height, width), grouped heads, an odd token count
        _rope("rope_video_grad", 1, 9999, 32, 8, 128, axes=3, inverse=True),
        # one decoding step of 64 sequences
        _paged("append_step_64", "append", 64, 1, 1500, 32, 8, 128, 16),
        # ragged prompts that enter the cache
        _paged("append_prompts", "append", 3, 4500, 8192, 32, 8, 128, 64),
        # image and text tokens into an 8-bit cache, pages that are no power of two
        _paged("append_e4m3_image", "append", 5, 611, 2000, 16, 4, 64, 48, e4m3=True, axes=3, interleaved=True),
        # one sequence's next token: latency
        _paged("decode_1x2k", "attend", 1, 1, 2000, 32, 8, 128, 16, ragged=False),
        # a batch's next tokens, ragged contexts
        _paged("decode_64x8k", "attend", 64, 1, 8192, 32, 8, 128, 64),
        # long contexts in an 8-bit cache
        _paged("decode_4x32k_e4m3", "attend", 4, 1, 32768, 32, 8, 128, 128, e4m3=True, ragged=False),
        # four draft tokens a sequence to verify, wide groups, odd pages
        _paged("verify_16x4", "attend", 16, 4, 5003, 16, 2, 128, 48),
        # a chunk of a long prompt
        _paged("chunk_2k_of_32k", "attend", 1, 2048, 32768, 32, 8, 128, 64, ragged=False),
        # chunks and single tokens in one batch, 64-wide heads, 8-bit cache
        _paged("mixed_16_e4m3", "attend", 16, 512, 4096, 16, 8, 64, 32, e4m3=True, single=0.6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["rope", "append", "attend", "attend", "attend"])
        D = rng.choice([64, 128])
        H_kv = rng.choice([1, 2, 4, 5, 8])
        H_q = H_kv * rng.choice([1, 2, 3, 4, 7, 8])
        if op == "rope":
            case = _rope("", rng.choice([1, 2, 3]), _log_int(rng, 16, 10000), H_q, H_kv, D, axes=rng.choice([1, 1, 3]),
                         inverse=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                         start=rng.choice([0, 0, _log_int(rng, 1, 1000000)]), rotated=rng.choice([D, D, D // 2]))
            ok = case["B"] * case["S"] * (H_q + H_kv) * D <= 2 * 8192 * 32 * 128
        elif op == "append":
            ctx = _log_int(rng, 16, 8192)
            new = rng.choice([1, rng.randint(1, 8), _log_int(rng, 1, ctx)])
            case = _paged("", op, _log_int(rng, 1, 64), min(new, ctx), ctx, H_q, H_kv, D,
                          16 * rng.choice([1, 2, 3, 4, 8]), e4m3=rng.random() < 0.4, single=rng.choice([0.0, 0.0, 0.5]),
                          axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.3)
            B = case["B"]
            ok = B * ctx * H_kv * D <= 2 ** 27 and B * case["new"] * (H_q + 2 * H_kv) * D <= 13500 * 48 * 128
        else:
            ctx = _log_int(rng, 16, 32768)
            new = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 1, 2048)])
            case = _paged("", op, _log_int(rng, 1, 64), min(new, ctx), ctx, H_q, H_kv, D,
                          16 * rng.choice([1, 2, 3, 4, 8]), e4m3=rng.random() < 0.4, single=rng.choice([0.0, 0.0, 0.5]),
                          causal=rng.random() < 0.85)
            B = case["B"]
            ok = (B * ctx * H_kv * D <= 2 ** 29 and B * case["new"] * H_q * ctx <= 2 ** 31
                  and B * case["new"] * H_q * ctx * 4 * D <= most)
        if ok:
            del case["name"]
            return case


def _lengths(case):
    """(new tokens, keys with them) of each sequence: a matter of the case, not of the seed."""
    r = random.Random("%(B)d %(new)d %(ctx)d %(single)s" % case)
    new, keys = [], []
    for b in range(case["B"]):
        n = 1 if b > 0 and r.random() < case["single"] else case["new"]
        if case["ragged"] and b > 0 and n > 1:
            n = r.randint((n + 1) // 2, n)
        new.append(n)
        keys.append(max(n, r.randint(case["ctx"] // 8, case["ctx"])) if case["ragged"] and b > 0 else case["ctx"])
    return new, keys


def _pairs(case):
    """Visible (query, key) pairs of one query head."""
    new, keys = _lengths(case)
    if not case["causal"]:
        return sum(n * k for n, k in zip(new, keys))
    return sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(new, keys))


def work(case):
    D, H_q, H_kv = case["D"], case["H_q"], case["H_kv"]
    if case["op"] == "rope":
        tokens = case["B"] * case["S"]
        moved = tokens * (H_q + H_kv) * D
        return {"bytes": 4 * moved + 4 * tokens * case["axes"], "flops": 3 * moved}
    new, keys = _lengths(case)
    tokens, cell = sum(new), 1 if case["e4m3"] else 2
    if case["op"] == "append":
        moved = tokens * (H_q + H_kv) * D
        return {"bytes": 2 * moved + 2 * tokens * H_kv * D + 2 * tokens * H_q * D + 2 * cell * tokens * H_kv * D
                + 4 * tokens * (case["axes"] if case["axes"] > 1 else 0), "flops": 3 * moved}
    return {"bytes": 2 * cell * sum(keys) * H_kv * D + 4 * tokens * H_q * D + 4 * tokens * H_q
            + 4 * sum(-(-k // case["page"]) for k in keys), "flops": 4 * D * H_q * _pairs(case)}


# ---------------------------------------------------------------------------------------------
# inputs

def _inv_freq(dims, base, dev):
    return (1.0 / base ** (torch.arange(0, dims, 2, dtype=torch.float64) / dims)).float().to(dev)


def _sections(axes, freqs):
    """Frequencies of each axis: a quarter for time, the rest for height and width alike."""
    if axes == 1:
        return (freqs,)
    t = freqs // 4
    h = (freqs - t) // 2
    return (t, h, freqs - t - h)


def _grid_positions(tokens, start, dev):
    """(time, height, width) of frames of 24 x 40 patches."""
    i = torch.arange(tokens, device=dev)
    return torch.stack([start + i // 960, start + i // 40 % 24, start + i % 40]).int()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    D, H_q, H_kv = case["D"], case["H_q"], case["H_kv"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {"case": dict(case)}
    if case["op"] == "rope":
        B, S = case["B"], case["S"]
        s["q"], s["k"] = normal(B, S, H_q, D).bfloat16(), normal(B, S, H_kv, D).bfloat16()
        s["inv_freq"] = _inv_freq(case["rotated"], 10000.0, dev)
        s["sections"] = _sections(case["axes"], case["rotated"] // 2)
        if case["axes"] > 1:
            s["positions"] = _grid_positions(B * S, case["start"], dev).view(3, B, S)
        else:
            s["positions"] = (case["start"] + torch.arange(S, device=dev, dtype=torch.int32)).expand(B, S).contiguous()
        if own:
            import attention_attn_fwd_10_b200 as attn

            s["rotary"] = attn.Rotary(s["inv_freq"], sections=s["sections"], interleaved=case["interleaved"])
        return s

    new, keys = _lengths(case)
    B, page, tokens = case["B"], case["page"], sum(new)
    pages = [-(-k // page) for k in keys]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).int()
    table = torch.zeros((B, max(pages)), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    s["page_table"] = table
    s["seq_len"] = torch.tensor(keys, dtype=torch.int32, device=dev)
    s["q_start"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    s["max_new"], s["max_keys"] = max(new), max(keys)
    s["k_scale"], s["v_scale"] = (0.03125, 0.02) if case["e4m3"] else (1.0, 1.0)

    def cache(x, scale):
        return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) if case["e4m3"] else x.bfloat16()

    # keys: some rows much larger than the others, as the first tokens of a text; values: channels with a mean of their own
    k = normal(n_pages, page, H_kv, D)
    k = k * torch.where(torch.rand((n_pages, page, H_kv, 1), generator=g, device=dev) < 0.01, 3.0, 1.0)
    s["k_cache"] = cache(k, s["k_scale"])
    del k
    s["v_cache"] = cache(normal(n_pages, page, H_kv, D) + 0.5 * normal(H_kv, D), s["v_scale"])
    s["q"] = (1.25 * normal(tokens, H_q, D)).bfloat16()
    if case["op"] == "append":
        s["k"], s["v"] = normal(tokens, H_kv, D).bfloat16(), normal(tokens, H_kv, D).bfloat16()
        s["inv_freq"] = _inv_freq(D, 500000.0, dev)
        s["sections"] = _sections(case["axes"], D // 2)
        # text: a token's position is its index in the sequence
        s["positions"] = _grid_positions(tokens, 17, dev) if case["axes"] > 1 else None
    if own:
        import attention_attn_fwd_10_b200 as attn

        s["cache"] = attn.PagedKV(s["k_cache"], s["v_cache"], s["page_table"], s["seq_len"], s["q_start"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"])
        if case["op"] == "append":
            s["rotary"] = attn.Rotary(s["inv_freq"], sections=s["sections"], interleaved=case["interleaved"])
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import attention_attn_fwd_10_b200 as attn

        if op == "rope":
            return attn.rope(s["q"], s["k"], rotary=s["rotary"], positions=s["positions"], inverse=s["case"]["inverse"])
        if op == "append":
            q = attn.paged_append(s["cache"], s["k"], s["v"], q=s["q"], rotary=s["rotary"], positions=s["positions"])
            return q, s["k_cache"], s["v_cache"]
        return attn.fwd_paged(s["cache"], s["q"], causal=s["case"]["causal"], max_new=s["max_new"])
    if op == "rope":
        cos, sin = _cos_sin(s["positions"].reshape(-1, *s["q"].shape[:2]), s["inv_freq"], s["sections"])
        sin = -sin if s["case"]["inverse"] else sin
        return tuple(_rotate(x, cos, sin, s["case"]["interleaved"]).to(x.dtype) for x in (s["q"], s["k"]))
    if op == "append":
        return _append_plain(s)
    return _attend_plain(s)


def _cos_sin(positions, inv_freq, sections):
    """positions [axes, ...] -> cos and sin [..., 1, frequencies] (angles in 64 bits: a far position's
    angle has no fraction left in 32)."""
    axis = torch.repeat_interleave(torch.arange(len(sections), device=inv_freq.device),
                                   torch.tensor(sections, device=inv_freq.device), output_size=inv_freq.numel())
    angle = positions.movedim(0, -1)[..., axis].double() * inv_freq.double()
    return angle.cos().float().unsqueeze(-2), angle.sin().float().unsqueeze(-2)


def _rotate(x, cos, sin, interleaved):
    n = cos.shape[-1]
    x = x.float()
    turned, rest = x[..., :2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = turned[..., :n], turned[..., n:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _owners(s):
    """Each new token's sequence, and its index among that sequence's keys."""
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    b = torch.searchsorted(s["q_start"], t.int(), right=True) - 1
    return b, s["seq_len"][b] - s["q_start"][b + 1] + t


def _append_plain(s):
    b, key = _owners(s)
    positions = key.unsqueeze(0) if s["positions"] is None else s["positions"]
    cos, sin = _cos_sin(positions, s["inv_freq"], s["sections"])
    page = s["page_table"][b, key // s["case"]["page"]].long()
    slot = key % s["case"]["page"]
    k, v = _rotate(s["k"], cos, sin, s["case"]["interleaved"]), s["v"].float()
    if s["case"]["e4m3"]:
        # bytes: the 8-bit type itself has no indexed store
        k = (k / s["k_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / s["v_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k_cache"].view(torch.uint8)[page, slot] = k
        s["v_cache"].view(torch.uint8)[page, slot] = v
    else:
        s["k_cache"][page, slot] = k.bfloat16()
        s["v_cache"][page, slot] = v.bfloat16()
    return _rotate(s["q"], cos, sin, s["case"]["interleaved"]).bfloat16(), s["k_cache"], s["v_cache"]


def _gather(cache, table, keys, scale):
    """[B, keys, H_kv, D] in 32 bits."""
    rows = cache.view(torch.uint8)[table.long()].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[table.long()]
    return rows.flatten(1, 2)[:, :keys].float() * scale


def _attend_plain(s):
    case = s["case"]
    q, D = s["q"], case["D"]
    (T, H_q, _), H_kv, B, n = q.shape, case["H_kv"], case["B"], s["max_new"]
    k = _gather(s["k_cache"], s["page_table"], s["max_keys"], s["k_scale"])
    v = _gather(s["v_cache"], s["page_table"], s["max_keys"], s["v_scale"])
    b, key = _owners(s)
    place = torch.arange(T, device=q.device) - s["q_start"][b]
    padded = torch.zeros((B, n, H_q, D), device=q.device)
    padded[b, place] = q.float()
    padded = padded.view(B, n, H_kv, H_q // H_kv, D).permute(0, 2, 3, 1, 4).reshape(B, H_kv, -1, D)  # [B, H_kv, G n, D]
    scores = (padded @ k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    # the last key that each new token sees
    last = torch.full((B, n), -1, device=q.device, dtype=key.dtype)
    last[b, place] = key if case["causal"] else s["seq_len"][b].to(key.dtype) - 1
    hidden = torch.arange(s["max_keys"], device=q.device) > last[:, :, None]  # [B, n, keys]
    scores.view(B, H_kv, -1, n, s["max_keys"]).masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    # keys past a sequence's end hold other sequences' values: finite, and of weight 0
    o = (weights @ v.transpose(1, 2)) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.view(B, H_kv, H_q // H_kv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H_q, D)[b, place]
    lse = lse.view(B, H_q, n)[b, :, place].t().contiguous()
    return o.bfloat16(), lse


# ---------------------------------------------------------------------------------------------
# the definition, in 64 bits

def _turn(x, positions, case, s):
    """x [..., H, D] turned, as complex numbers; positions: one tensor for each axis."""
    n = s["inv_freq"].numel()
    angle = torch.cat([p.double()[..., None] * f.double() for p, f in zip(positions, s["inv_freq"].split(list(s["sections"])))], -1)
    if case.get("inverse"):
        angle = -angle
    x = x.double().clone()
    re, im = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if case["interleaved"] else (x[..., :n], x[..., n:2 * n])
    z = torch.complex(re.contiguous(), im.contiguous()) * torch.polar(torch.ones_like(angle), angle)[..., None, :]
    re.copy_(z.real)
    im.copy_(z.imag)
    return x


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        positions = s["positions"].reshape(-1, case["B"], case["S"]).unbind(0)
        return _turn(s["q"], positions, case, s), _turn(s["k"], positions, case, s)
    new, keys = _lengths(case)
    page, table = case["page"], s["page_table"].cpu()
    if case["op"] == "append":
        index = torch.cat([torch.arange(n_k - n, n_k) for n, n_k in zip(new, keys)]).to(s["q"].device)
        positions = [index] if s["positions"] is None else list(s["positions"].unbind(0))
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k, v = _turn(s["k"], positions, case, s) / s["k_scale"], s["v"].double() / s["v_scale"]
        if case["e4m3"]:
            k, v = k.clamp(-E4M3_MAX, E4M3_MAX), v.clamp(-E4M3_MAX, E4M3_MAX)
        t = 0
        for b, (n, n_k) in enumerate(zip(new, keys)):
            i = torch.arange(n_k - n, n_k)
            rows = (table[b][i // page].long() * page + i % page).to(k.device)
            k_cache.flatten(0, 1)[rows] = k[t:t + n]
            v_cache.flatten(0, 1)[rows] = v[t:t + n]
            t += n
        return _turn(s["q"], positions, case, s), k_cache, v_cache
    group = case["H_q"] // case["H_kv"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty((case["H_q"], s["q"].shape[0]), dtype=torch.float64, device=s["q"].device)
    t = 0
    for b, (n, n_k) in enumerate(zip(new, keys)):
        i = torch.arange(n_k)
        rows = (table[b][i // page].long() * page + i % page).to(o.device)
        k_all, v_all = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
        if case["e4m3"]:
            k_all, v_all = k_all.view(torch.uint8), v_all.view(torch.uint8)
        k_b = k_all[rows].view(s["k_cache"].dtype).double() * s["k_scale"]
        v_b = v_all[rows].view(s["v_cache"].dtype).double() * s["v_scale"]
        seen = torch.ones((n, n_k), dtype=torch.bool, device=o.device)
        if case["causal"]:
            seen = seen.tril(n_k - n)
        for h in range(case["H_q"]):
            x = s["q"][t:t + n, h].double() @ k_b[:, h // group].T / math.sqrt(case["D"])
            x = x.masked_fill(~seen, -math.inf)
            lse[h, t:t + n] = torch.logsumexp(x, -1)
            o[t:t + n, h] = torch.exp(x - lse[h, t:t + n, None]) @ v_b[:, h // group]
        t += n
    return o, lse
