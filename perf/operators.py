"""The operators around the selection of a sparse-attention step: rotary positions, the indexer's
scores over a paged key cache, and attention over the selected entries of a paged cache.

`run` computes them in their plain form (elementary torch operations in 32 bits) or, where `own` is
true, through this package's calls. `exact` is the definition in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ---- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # A decode step of four sequences: the queries of 64 heads, half of each head rotated.
        dict(name="rotary_decode", op="rotary", T=4, H=64, D=128, rotated=64, offset=0, layout="half", type="bf16",
             scaling=1.0, inverse=False, extra_heads=0, page_size=0),
        # A prompt's queries at far positions, frequencies scaled for a long context, the head's second half rotated.
        dict(name="rotary_prompt", op="rotary", T=8192, H=64, D=128, rotated=64, offset=64, layout="interleaved",
             type="bf16", scaling=16.0, inverse=False, extra_heads=0, page_size=0),
        # A chunk of prompt keys rotated on their way into the paged cache.
        dict(name="rotary_append", op="rotary", T=1000, H=8, D=128, rotated=128, offset=0, layout="half", type="fp16",
             scaling=1.0, inverse=False, extra_heads=0, page_size=64),
        # The backward rotation of fp32 gradients that lie inside a joint query-key-value tensor; odd sizes.
        dict(name="rotary_inverse", op="rotary", T=4097, H=24, D=80, rotated=80, offset=0, layout="interleaved",
             type="fp32", scaling=1.0, inverse=True, extra_heads=12, page_size=0),
        # The latency batch: four rows of 0 to 8192 keys.
        dict(name="scores_decode_small", op="scores", B=4, T=1, H=64, D=128, S=8192, lengths="latency", page_size=64,
             type="bf16"),
        # A decode batch of long ragged rows.
        dict(name="scores_decode_long", op="scores", B=64, T=1, H=64, D=128, S=65536, lengths="ragged", page_size=64,
             type="bf16"),
        # A prompt's last 2048 tokens against its 8192 keys.
        dict(name="scores_prefill", op="scores", B=1, T=2048, H=64, D=128, S=8192, lengths="causal", page_size=64,
             type="bf16"),
        # 8-bit keys with a scale for each, two tokens a sequence (the second one speculated), odd width.
        dict(name="scores_e4m3_two_tokens", op="scores", B=32, T=2, H=32, D=128, S=32769, lengths="ragged",
             page_size=16, type="e4m3"),
        # A small decode batch: latency.
        dict(name="attention_decode_small", op="attention", B=4, T=1, Hq=32, Hkv=4, D=128, Dv=128, K=512, S=8192,
             page_size=64, type="bf16", shared=False, cap=0.0, bias=False, documents=False),
        # A decode batch, capped scores, the widest selection.
        dict(name="attention_decode_capped", op="attention", B=64, T=1, Hq=64, Hkv=8, D=128, Dv=128, K=2048, S=16384,
             page_size=64, type="bf16", shared=False, cap=30.0, bias=False, documents=False),
        # A prompt's last 2048 tokens, one latent entry a token that holds keys and values.
        dict(name="attention_prefill_shared", op="attention", B=1, T=2048, Hq=64, Hkv=1, D=256, Dv=192, K=512, S=8192,
             page_size=64, type="bf16", shared=True, cap=0.0, bias=False, documents=False),
        # Three tokens a sequence, odd heads, pages and width, a distance bias and packed documents.
        dict(name="attention_biased_odd", op="attention", B=16, T=3, Hq=40, Hkv=5, D=96, Dv=64, K=1000, S=32769,
             page_size=17, type="fp16", shared=False, cap=0.0, bias=True, documents=True),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotary", "scores", "attention"])
    if op == "rotary":
        D = 8 * _spread(rng, 4, 32)
        H = _spread(rng, 1, 96)
        T = _spread(rng, 1, max(2, 8192 * 64 * 128 // (2 * H * D)))
        rotated = min(D, 16 * _spread(rng, 1, max(1, D // 16)))
        return dict(op=op, T=T, H=H, D=D, rotated=rotated, offset=rng.choice([0, (D - rotated) // 8 * 8]),
                    layout=rng.choice(["half", "interleaved"]), type=rng.choice(["bf16", "fp16", "fp32"]),
                    scaling=rng.choice([1.0, 4.0, 16.0]), inverse=rng.random() < 0.3,
                    extra_heads=rng.choice([0, 0, 3]), page_size=rng.choice([0, 0, 16, 48, 64]))
    if op == "scores":
        H = rng.choice([1, 8, 16, 24, 32, 48, 64, 64])
        S = _spread(rng, 100, 65536)
        if rng.random() < 0.6:
            B, T = _spread(rng, 1, max(1, min(256, 64 * 65536 // S))), rng.choice([1, 1, 2, 3])
            T = min(T, max(1, 64 * 65536 // (B * S)))
            lengths = "ragged"
        else:
            B, T, lengths = rng.choice([1, 1, 2]), _spread(rng, 16, max(16, min(2048, 2048 * 8192 // (2 * S)))), "causal"
        return dict(op=op, B=B, T=T, H=H, D=rng.choice([64, 128, 128]), S=S, lengths=lengths,
                    page_size=rng.choice([1, 16, 48, 64, 64, 256]), type=rng.choice(["bf16", "bf16", "fp16", "e4m3"]))
    Hkv = rng.choice([1, 2, 4, 5, 8])
    Hq = Hkv * rng.choice([1, 4, 7, 8, 16, 128 if Hkv == 1 else 8])
    D = rng.choice([64, 96, 128, 128, 192, 256])
    shared = Hkv == 1 and rng.random() < 0.5
    Dv = min(D, rng.choice([64, 128, 256])) if shared else rng.choice([64, 128, D])
    K = _spread(rng, 1, 2048)
    S = max(K, _spread(rng, 100, 32768))
    rows = _spread(rng, 1, max(1, min(1024, 64 * 2048 * 8 * 256 // (2 * K * Hkv * (D + Dv)))))
    T = rng.choice([1, 1, 2, 3, rows])
    B = max(1, min(rows // T, 64 * 16384 * 8 * 256 // (2 * S * Hkv * (D + Dv))))
    return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, Dv=Dv, K=K, S=S, page_size=rng.choice([1, 16, 48, 64, 64]),
                type=rng.choice(["bf16", "bf16", "fp16"]), shared=shared, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                bias=rng.random() < 0.3, documents=rng.random() < 0.3)


# ---- inputs -----------------------------------------------------------------------------------------


def _frequencies(rotated, scaling, device):
    """Radians per position of each pair, in 64 bits; `scaling` stretches the long waves as a linear ramp over the
    pairs (the far half is divided by it), the way a context is lengthened."""
    i = torch.arange(rotated // 2, dtype=torch.float64, device=device)
    f = 10000.0 ** (-2.0 * i / rotated)
    ramp = (i / max(1, rotated // 2 - 1)).clamp(0.0, 1.0)
    return f * (1.0 - ramp) + f / scaling * ramp


def _pool(B, S, page_size, gen, device):
    """A page table [B, pages]: the pages of all sequences are one random permutation of the pool."""
    pages = -(-S // page_size)
    return torch.randperm(B * pages, generator=gen, device=device).to(torch.int32).view(B, pages)


def _lengths(case, gen, device):
    B, T, S = case["B"], case["T"], case["S"]
    if case["lengths"] == "latency":
        last = torch.tensor([0, 300, 512, 8192], device=device)[:B]
    elif case["lengths"] == "causal":
        last = torch.full((B,), S, device=device)
    else:
        last = torch.randint(int(0.8 * S), S + 1, (B,), generator=gen, device=device)
    back = torch.arange(T - 1, -1, -1, device=device)
    return (last[:, None] - back).clamp(min=0).to(torch.int32)


def _prepare_rotary(case, gen, device):
    T, H, D, t = case["T"], case["H"], case["D"], _TYPES[case["type"]]
    joint = torch.randn((T, H + case["extra_heads"], D), generator=gen, device=device).to(t)
    state = dict(case=case, x=joint[:, :H], layout=case["layout"], offset=case["offset"], inverse=case["inverse"],
                 positions=torch.randint(0, 1 << 20, (T,), generator=gen, device=device).to(torch.int32),
                 frequencies=_frequencies(case["rotated"], case["scaling"], device),
                 scale=1.0 if case["scaling"] == 1.0 else 0.1 * math.log(case["scaling"]) + 1.0, cache=None)
    if case["page_size"]:
        ps = case["page_size"]
        pages = -(-T // ps) + 2
        state["cache"] = torch.zeros((pages, ps, H, D), dtype=t, device=device)
        state["slots"] = torch.randperm(pages * ps, generator=gen, device=device)[:T].to(torch.int32)
        state["slots"][3::7] = -1  # tokens that this cache does not keep
    else:
        state["out"] = torch.empty((T, H, D), dtype=t, device=device)
    return state


def _prepare_scores(case, gen, device):
    B, T, H, D, S, t = case["B"], case["T"], case["H"], case["D"], case["S"], _TYPES[case["type"]]
    table = _pool(B, S, case["page_size"], gen, device)
    keys = torch.randn((table.numel(), case["page_size"], D), generator=gen, device=device, dtype=torch.bfloat16)
    scales = None
    if case["type"] == "e4m3":
        scales = torch.rand((table.numel(), case["page_size"]), generator=gen, device=device) * 0.02 + 0.005
        keys = keys.mul_(64.0).clamp_(-448.0, 448.0)
    q = torch.randn((B, T, H, D), generator=gen, device=device)
    weights = torch.randn((B, T, H), generator=gen, device=device) / math.sqrt(H * D)
    return dict(case=case, q=q.to(t), weights=weights, keys=keys.to(t), key_scales=scales, table=table,
                lengths=_lengths(case, gen, device), out=torch.zeros((B, T, S), dtype=torch.float32, device=device))


def _prepare_attention(case, gen, device):
    B, T, Hq, Hkv, D, Dv, K, S = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "Dv", "K", "S"))
    t, ps = _TYPES[case["type"]], case["page_size"]
    table = _pool(B, S, ps, gen, device)
    k = torch.randn((table.numel(), ps, Hkv, D), generator=gen, device=device, dtype=t)
    v = k[..., :Dv] if case["shared"] else torch.randn((table.numel(), ps, Hkv, Dv), generator=gen, device=device,
                                                       dtype=t)
    last = torch.randint(int(0.8 * S), S + 1, (B,), generator=gen, device=device)
    qpos = (last[:, None] - T + torch.arange(T, device=device)).clamp(min=0)
    # the selection: distinct positions up to the query's own, ascending, -1 after the last
    r = torch.rand((B, T, S), generator=gen, device=device)
    r.masked_fill_(torch.arange(S, device=device) > qpos[..., None], -1.0)
    best, picked = r.topk(K, dim=-1, sorted=False)
    picked = picked.masked_fill(best < 0, S).sort(dim=-1).values
    indices = picked.masked_fill(picked == S, -1).to(torch.int32)
    if B * T > 4:
        indices[0, 0] = -1  # an idle row
    state = dict(case=case, q=(torch.randn((B, T, Hq, D), generator=gen, device=device) * 1.5).to(t), k=k, v=v,
                 indices=indices, table=table, qpos=qpos.to(torch.int32), scale=1.0 / math.sqrt(D), cap=case["cap"],
                 slopes=None, first=None)
    if case["bias"]:
        state["slopes"] = 2.0 ** (-8.0 * (torch.arange(Hq, device=device, dtype=torch.float32) + 1) / Hq)
    if case["documents"]:
        state["first"] = (qpos.double() * torch.rand((B, T), generator=gen, device=device)).to(torch.int32)
    return state


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    return {"rotary": _prepare_rotary, "scores": _prepare_scores, "attention": _prepare_attention}[case["op"]](
        case, gen, device)


# ---- the plain forms --------------------------------------------------------------------------------


def _rotary_plain(state):
    x, case = state["x"], state["case"]
    R, offset = case["rotated"], state["offset"]
    angle = state["positions"].double()[:, None] * state["frequencies"]
    cos = (torch.cos(angle) * state["scale"]).float()[:, None]
    sin = (torch.sin(angle) * state["scale"]).float()[:, None]
    if state["inverse"]:
        sin = -sin
    part = x[..., offset:offset + R].float()
    if state["layout"] == "half":
        a, b = part[..., :R // 2], part[..., R // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    y = torch.cat([x[..., :offset], turned.to(x.dtype), x[..., offset + R:]], dim=-1)
    if state["cache"] is None:
        return y
    # a token that is not kept writes the first one's row once more
    row = torch.where(state["slots"] >= 0, torch.arange(case["T"], device=y.device), 0)
    state["cache"].flatten(0, 1)[state["slots"].long()[row]] = y[row]
    return state["cache"]


def _positions_to_slots(table, positions, page_size):
    """Slots of positions [B, T, n] (or [B, n]) of each sequence; negative positions stand for slot 0."""
    p = positions.clamp(min=0).long()
    pages = torch.gather(table.long(), 1, (p // page_size).flatten(1)).view(p.shape)
    return pages * page_size + p % page_size


def _scores_plain(state):
    case = state["case"]
    B, S = case["B"], case["S"]
    s = torch.arange(S, device=state["q"].device)
    slots = _positions_to_slots(state["table"], s.expand(B, S), case["page_size"])
    keys = state["keys"].flatten(0, 1)[slots].float()
    dots = torch.matmul(state["q"].flatten(1, 2).float(), keys.transpose(1, 2)).clamp_(min=0)
    dots = dots.view(B, case["T"], case["H"], S)
    scores = torch.matmul(state["weights"][:, :, None, :], dots)[:, :, 0]
    if state["key_scales"] is not None:
        scores = scores * state["key_scales"].flatten()[slots][:, None]
    return torch.where(s < state["lengths"][..., None], scores, state["out"], out=state["out"])


def _attention_plain(state):
    case = state["case"]
    B, T, Hq, Hkv, K = (case[n] for n in ("B", "T", "Hq", "Hkv", "K"))
    pos = state["indices"]
    slots = _positions_to_slots(state["table"], pos, case["page_size"])
    k = state["k"].flatten(0, 1)[slots].float()
    v = state["v"].flatten(0, 1)[slots].float()
    q = state["q"].float().view(B, T, Hkv, Hq // Hkv, -1)
    z = torch.matmul(q, k.permute(0, 1, 3, 4, 2)) * state["scale"]
    if state["cap"]:
        z = state["cap"] * torch.tanh(z / state["cap"])
    away = (pos - state["qpos"][..., None]).float()
    if state["slopes"] is not None:
        z = z + state["slopes"].view(Hkv, -1, 1) * away[:, :, None, None]
    seen = (pos >= 0) & (away <= 0)
    if state["first"] is not None:
        seen = seen & (pos >= state["first"][..., None])
    z = z.masked_fill(~seen[:, :, None, None], -math.inf)
    top = z.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(z - top)
    total = e.sum(dim=-1, keepdim=True)
    out = torch.matmul(e, v.transpose(2, 3)) / total.clamp(min=1e-37)
    lse = torch.log(total) + top
    return out.view(B, T, Hq, -1).to(state["q"].dtype), lse.view(B, T, Hq)


# ---- one pass ---------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rotary": _rotary_plain, "scores": _scores_plain, "attention": _attention_plain}[op](state)
    import sparse_attention_indexer_fp32_gb300 as tk

    if op == "rotary":
        if state["cache"] is not None:
            return tk.rotary(state["x"], state["positions"], state["frequencies"], layout=state["layout"],
                             offset=state["offset"], scale=state["scale"], inverse=state["inverse"],
                             out=state["cache"], slots=state["slots"])
        return tk.rotary(state["x"], state["positions"], state["frequencies"], layout=state["layout"],
                         offset=state["offset"], scale=state["scale"], inverse=state["inverse"], out=state["out"])
    if op == "scores":
        return tk.indexer_scores(state["q"], state["weights"], state["keys"], state["lengths"], state["table"],
                                 key_scales=state["key_scales"], out=state["out"])
    return tk.sparse_attention(state["q"], state["k"], state["v"], state["indices"], state["table"],
                               query_positions=state["qpos"], scale=state["scale"], softcap=state["cap"],
                               slopes=state["slopes"], first=state["first"], return_lse=True)


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    b = _BYTES[case["type"]]
    if case["op"] == "rotary":
        T, H, D = case["T"], case["H"], case["D"]
        kept = 6 / 7 if case["page_size"] and T > 7 else 1.0
        return {"bytes": int(2 * kept * T * H * D * b) + 4 * T, "flops": int(3 * kept * T * H * case["rotated"])}
    B, T, S, D = case["B"], case["T"], case["S"], case["D"]
    if case["op"] == "scores":
        if case["lengths"] == "latency":
            keys = pairs = 0 + 300 + 512 + 8192
        elif case["lengths"] == "causal":
            keys, pairs = B * S, B * sum(max(0, S - i) for i in range(T))
        else:
            keys = int(0.9 * B * S)
            pairs = keys * T
        scale = 4 * keys if case["type"] == "e4m3" else 0
        return {"bytes": keys * D * b + scale + 4 * pairs + B * T * case["H"] * (D * b + 4) + 4 * keys // case["page_size"],
                "flops": 2 * pairs * case["H"] * (D + 1)}
    Hq, Hkv, Dv, K = case["Hq"], case["Hkv"], case["Dv"], case["K"]
    part = 0.5 if case["documents"] else 1.0
    chosen = int(part * B * T * min(K, int(0.9 * S)))
    entries = min(chosen, int(part * 0.9 * B * S))
    entry = Hkv * (D if case["shared"] else D + Dv) * b
    return {"bytes": entries * entry + 4 * B * T * K + B * T * Hq * ((D + Dv) * b + 4),
            "flops": 2 * chosen * Hq * (D + Dv)}


# ---- the definition in 64 bits ----------------------------------------------------------------------


def _exact_rotary(s, case):
    x = s["x"].double()
    R, o = case["rotated"], case["offset"]
    turn = s["positions"].double().view(-1, 1, 1) * s["frequencies"].view(1, 1, -1)
    if case["inverse"]:
        turn = -turn
    z = torch.polar(torch.full_like(turn, s["scale"]), turn)
    if case["layout"] == "half":
        first, second = slice(o, o + R // 2), slice(o + R // 2, o + R)
    else:
        first, second = slice(o, o + R, 2), slice(o + 1, o + R, 2)
    w = torch.complex(x[..., first], x[..., second]) * z
    y = x.clone()
    y[..., first], y[..., second] = w.real, w.imag
    if s["cache"] is None:
        return y
    pages, ps = s["cache"].shape[:2]
    flat = torch.zeros((pages * ps + 1,) + tuple(y.shape[1:]), dtype=torch.float64, device=y.device)
    where = s["slots"].long()
    flat[torch.where(where < 0, pages * ps, where)] = y
    return flat[:-1].view(s["cache"].shape)


def _exact_scores(s, case):
    B, T, S, ps = case["B"], case["T"], case["S"], case["page_size"]
    out = torch.zeros((B, T, S), dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        order = s["table"][b].long()
        keys = s["keys"][order].reshape(-1, case["D"])[:S].double()
        if s["key_scales"] is not None:
            keys = keys * s["key_scales"][order].reshape(-1, 1)[:S].double()
        for t0 in range(0, T, 256):
            q = s["q"][b, t0:t0 + 256].double()
            dots = torch.relu(torch.einsum("thd,sd->ths", q, keys))
            got = torch.einsum("th,ths->ts", s["weights"][b, t0:t0 + 256].double(), dots)
            n = s["lengths"][b, t0:t0 + 256].long()
            keep = torch.arange(S, device=got.device)[None] < n[:, None]
            out[b, t0:t0 + 256] = torch.where(keep, got, 0.0)
    return out


def _exact_attention(s, case):
    B, T, Hq, Hkv, ps = (case[n] for n in ("B", "T", "Hq", "Hkv", "page_size"))
    out = torch.zeros((B, T, Hq, case["Dv"]), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    head = torch.arange(Hq, device=s["q"].device) // (Hq // Hkv)
    for b in range(B):
        for t0 in range(0, T, 16):
            idx = s["indices"][b, t0:t0 + 16].long()
            safe = idx.clamp(min=0)
            page = s["table"][b].long()[safe // ps]
            k = s["k"][page, safe % ps].double()
            v = s["v"][page, safe % ps].double()
            q = s["q"][b, t0:t0 + 16].double()
            z = torch.einsum("thd,tkhd->thk", q, k.index_select(2, head)) * s["scale"]
            if s["cap"]:
                z = s["cap"] * torch.tanh(z / s["cap"])
            now = s["qpos"][b, t0:t0 + 16].long()[:, None]
            if s["slopes"] is not None:
                z = z + s["slopes"].double()[None, :, None] * (idx - now).double()[:, None]
            hidden = (idx < 0) | (idx > now)
            if s["first"] is not None:
                hidden = hidden | (idx < s["first"][b, t0:t0 + 16].long()[:, None])
            z = z.masked_fill(hidden[:, None], -math.inf)
            lse[b, t0:t0 + 16] = torch.logsumexp(z, dim=-1)
            p = torch.nan_to_num(torch.softmax(z, dim=-1), nan=0.0)
            out[b, t0:t0 + 16] = torch.einsum("thk,tkhd->thd", p, v.index_select(2, head))
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "scores": _exact_scores, "attention": _exact_attention}[case["op"]](s, case)
