"""The operators of a paged cache held in 8 bits: keys and values appended to it, the keys rotated on the way,
with a scale for each block of tokens and head that grows with what the block holds; and attention over
selected entries of such a cache. Appending to a 16-bit cache goes through the same call.

`run` computes them in their plain form (elementary torch operations in 32 bits) or, where `own` is
true, through this package's calls. `exact` is the definition in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_E4M3 = torch.float8_e4m3fn


# ---- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # A decode step of 64 sequences: a token each, into blocks that hold earlier tokens.
        dict(name="append_decode", op="append", B=64, n=1, spare=0, H=8, D=128, Dv=128, rotated=64, offset=0,
             layout="half", page_size=64, block=64, type="bf16"),
        # The prompts of four sequences, whole pages with a scale each.
        dict(name="append_prompt", op="append", B=4, n=2048, spare=0, H=8, D=128, Dv=128, rotated=128, offset=0,
             layout="half", page_size=64, block=64, type="bf16"),
        # A padded batch of three prompts' chunks in fp32: odd heads and sizes, short blocks, the rest of the batch idle.
        dict(name="append_padded_odd", op="append", B=3, n=1365, spare=2, H=5, D=112, Dv=80, rotated=48, offset=64,
             layout="interleaved", page_size=48, block=16, type="fp32"),
        # The indexer's keys: one head, a scale for each token, no values.
        dict(name="append_index_keys", op="append", B=2, n=4096, spare=0, H=1, D=128, Dv=0, rotated=64, offset=0,
             layout="half", page_size=64, block=1, type="bf16"),
        # Keys and values into a cache of the inputs' own type, prompt chunks of 16 sequences.
        dict(name="append_16bit", op="append", B=16, n=250, spare=7, H=8, D=128, Dv=128, rotated=128, offset=0,
             layout="half", page_size=64, block=0, type="fp16"),
        # A small decode batch: latency.
        dict(name="attention_decode_small", op="attention", B=4, T=1, Hq=32, Hkv=4, D=128, Dv=128, K=512, S=8192,
             page_size=64, block=64, type="bf16", shared=False, cap=0.0, bias=False, documents=False),
        # A decode batch, the widest selection.
        dict(name="attention_decode", op="attention", B=64, T=1, Hq=64, Hkv=8, D=128, Dv=128, K=2048, S=16384,
             page_size=64, block=64, type="bf16", shared=False, cap=0.0, bias=False, documents=False),
        # The same cache with capped logits, two tokens a sequence (the second one speculated), a scale for 16 tokens.
        dict(name="attention_two_capped", op="attention", B=32, T=2, Hq=64, Hkv=8, D=128, Dv=128, K=1024, S=16384,
             page_size=64, block=16, type="fp16", shared=False, cap=30.0, bias=False, documents=False),
        # A prompt's last 2048 tokens, one latent entry a token that holds keys and values, a scale for each.
        dict(name="attention_prefill_shared", op="attention", B=1, T=2048, Hq=64, Hkv=1, D=256, Dv=192, K=512, S=8192,
             page_size=64, block=1, type="bf16", shared=True, cap=0.0, bias=False, documents=False),
        # Three tokens a sequence, odd heads, pages and width, a distance bias and packed documents.
        dict(name="attention_biased_odd", op="attention", B=16, T=3, Hq=40, Hkv=5, D=96, Dv=64, K=1000, S=32769,
             page_size=51, block=17, type="fp16", shared=False, cap=0.0, bias=True, documents=True),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    if rng.random() < 0.5:
        H = _spread(rng, 1, 16)
        D, Dv = 8 * _spread(rng, 4, 32), rng.choice([0, 8 * _spread(rng, 4, 32), 128])
        T = _spread(rng, 1, max(2, 8192 * 8 * 256 // (H * (D + Dv) * 2)))
        n = rng.choice([1, 1, T, _spread(rng, 1, T)])
        rotated = min(D, 16 * _spread(rng, 1, max(1, D // 16)))
        page_size, block = rng.choice([(64, 64), (64, 16), (64, 1), (16, 16), (48, 8), (256, 128), (17, 17), (64, 0), (1, 0)])
        B = max(1, min(T // n, (1 << 25) // (page_size * H * (D + Dv))))  # sequences of one token: a page each
        return dict(op="append", B=B, n=n, spare=rng.choice([0, 0, 1, 5]), H=H, D=D, Dv=Dv, rotated=rotated,
                    offset=rng.choice([0, (D - rotated) // 8 * 8]), layout=rng.choice(["half", "interleaved"]),
                    page_size=page_size, block=block, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    Hkv = rng.choice([1, 2, 4, 5, 8])
    Hq = Hkv * rng.choice([1, 4, 7, 8, 16, 24, 100 if Hkv == 1 else 8])
    D = rng.choice([64, 96, 128, 128, 192, 256])
    shared = Hkv == 1 and rng.random() < 0.5
    Dv = min(D, rng.choice([64, 128, 256])) if shared else rng.choice([64, 128, D])
    K = _spread(rng, 1, 2048)
    S = max(K, _spread(rng, 100, 32768))
    page_size, block = rng.choice([(64, 64), (64, 64), (64, 16), (64, 1), (48, 8), (1, 1), (17, 17), (256, 128)])
    rows = _spread(rng, 1, max(1, min(1024, 64 * 2048 * 8 * 256 // (2 * K * Hkv * (D + Dv)))))
    T = rng.choice([1, 1, 2, 3, rows])
    B = max(1, min(rows // T, 64 * 16384 * 8 * 256 // (2 * S * Hkv * (D + Dv))))
    return dict(op="attention", B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, Dv=Dv, K=K, S=S, page_size=page_size, block=block,
                type=rng.choice(["bf16", "bf16", "fp16"]), shared=shared, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                bias=rng.random() < 0.3, documents=rng.random() < 0.3)


# ---- inputs -----------------------------------------------------------------------------------------


def _codes(shape, gen, device):
    """8-bit entries as a quantised cache holds them: the largest of a block near the type's largest value."""
    return torch.randn(shape, generator=gen, device=device, dtype=torch.bfloat16).mul_(110.0).clamp_(-448.0, 448.0).to(_E4M3)


def _prepare_append(case, gen, device):
    B, n, H, D, Dv, ps, t = (case[i] for i in ("B", "n", "H", "D", "Dv", "page_size", "type"))
    t = _TYPES[t]
    T = B * n + case["spare"]
    # sequence b goes on from a far position of its own; its pages, from the one it stands in, lie anywhere in the pool
    start = torch.randint(0, 1 << 20, (B,), generator=gen, device=device)
    pages = (n + ps - 2) // ps + 1
    table = torch.randperm(B * pages, generator=gen, device=device).view(B, pages)
    where = torch.arange(n, device=device) + (start % ps)[:, None]
    slots = torch.gather(table, 1, where // ps) * ps + where % ps
    # tokens behind the last sequence belong to none
    slots = torch.cat([slots.flatten(), torch.full((case["spare"],), -1, device=device)]).to(torch.int32)
    positions = (start[:, None] + torch.arange(n, device=device)).flatten()
    positions = torch.cat([positions, torch.zeros(case["spare"], dtype=positions.dtype, device=device)]).to(torch.int32)
    i = torch.arange(case["rotated"] // 2, dtype=torch.float64, device=device)
    state = dict(case=case, positions=positions, slots=slots, frequencies=10000.0 ** (-2.0 * i / case["rotated"]))
    # heads of different sizes: some outgrow the scale that their block has
    joint = torch.randn((T, H, D + Dv), generator=gen, device=device)
    joint *= torch.exp2(torch.randint(-2, 3, (H, 1), generator=gen, device=device).float())
    joint = joint.to(t)
    state["k"], state["v"] = joint[..., :D], joint[..., D:] if Dv else None
    for side, d in (("k", D), ("v", Dv)):
        shape = (B * pages, ps, H, d)
        if not d:
            state[side + "_cache"] = state[side + "_scales"] = None
        elif case["block"]:
            state[side + "_cache"] = _codes(shape, gen, device)
            exponent = torch.randint(-8, -5, (B * pages, ps // case["block"], H), generator=gen, device=device)
            state[side + "_scales"] = torch.exp2(exponent.float())
        else:
            state[side + "_cache"], state[side + "_scales"] = torch.zeros(shape, dtype=t, device=device), None
    return state


def _prepare_attention(case, gen, device):
    B, T, Hq, Hkv, D, Dv, K, S = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "Dv", "K", "S"))
    ps, blocks = case["page_size"], case["page_size"] // case["block"]
    pages = -(-S // ps)
    # the pages of all sequences are one random permutation of the pool
    table = torch.randperm(B * pages, generator=gen, device=device).to(torch.int32).view(B, pages)
    k = _codes((B * pages, ps, Hkv, D), gen, device)
    v = k[..., :Dv] if case["shared"] else _codes((B * pages, ps, Hkv, Dv), gen, device)
    k_scales = torch.exp2(torch.rand((B * pages, blocks, Hkv), generator=gen, device=device) * 2.0 - 8.0)
    v_scales = k_scales if case["shared"] else torch.exp2(
        torch.rand((B * pages, blocks, Hkv), generator=gen, device=device) * 2.0 - 8.0)
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
    q = (torch.randn((B, T, Hq, D), generator=gen, device=device) * 1.5).to(_TYPES[case["type"]])
    state = dict(case=case, q=q, k=k, v=v, k_scales=k_scales, v_scales=v_scales, indices=indices, table=table,
                 qpos=qpos.to(torch.int32), scale=1.0 / math.sqrt(D), cap=case["cap"], slopes=None, first=None)
    if case["bias"]:
        state["slopes"] = 2.0 ** (-8.0 * (torch.arange(Hq, device=device, dtype=torch.float32) + 1) / Hq)
    if case["documents"]:
        state["first"] = (qpos.double() * torch.rand((B, T), generator=gen, device=device)).to(torch.int32)
    return state


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    return {"append": _prepare_append, "attention": _prepare_attention}[case["op"]](case, gen, device)


# ---- the plain forms --------------------------------------------------------------------------------


def _turned(state):
    """The rotated keys in 32 bits, the angles in 64; and what bounds them at any angle: the sum of each pair's sizes."""
    case, x = state["case"], state["k"].float()
    R, offset = case["rotated"], case["offset"]
    angle = state["positions"].double()[:, None] * state["frequencies"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    part = x[..., offset:offset + R]
    if case["layout"] == "half":
        a, b = part[..., :R // 2], part[..., R // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    rest = (x[..., :offset], x[..., offset + R:])
    return torch.cat([rest[0], turned, rest[1]], dim=-1), torch.cat([rest[0].abs(), a.abs() + b.abs(), rest[1].abs()], dim=-1)


def _store(state, side, y, sizes):
    """Tokens into one cache; a token that is not kept writes the first one's entry once more."""
    cache, scales, slots, block = state[side + "_cache"], state[side + "_scales"], state["slots"].long(), state["case"]["block"]
    row = torch.where(slots >= 0, torch.arange(slots.numel(), device=slots.device), 0)
    if scales is None:
        cache.flatten(0, 1)[slots[row]] = y[row].to(cache.dtype)
        return
    H, D = cache.shape[2:]
    entries, old = cache.view(-1, block, H, D), scales.view(-1, H)
    to, place = slots[row] // block, slots[row] % block
    peak = torch.zeros_like(old).scatter_reduce(0, to[:, None].expand(-1, H), sizes[row].amax(dim=-1), "amax")
    first = torch.full((old.shape[0],), block, device=slots.device).scatter_reduce(0, to, place, "amin")[:, None]
    mantissa, exponent = torch.frexp(peak)  # the smallest power of two that brings it to 448 = 0.875 * 2^9 or below
    need = torch.exp2((exponent - 9 + (mantissa > 0.875)).clamp(min=-126).float())
    new = torch.where(first == block, old, torch.where(first == 0, need, torch.maximum(old, need)))
    held = torch.arange(block, device=slots.device)[None, :, None] < torch.where(first == block, 0, first)[:, None]
    again = (entries.float() * (old / new)[:, None, :, None]).clamp(-448.0, 448.0).to(_E4M3)
    entries.view(torch.uint8).copy_(torch.where(held[..., None], again.view(torch.uint8), entries.view(torch.uint8)))
    scales.view(-1, H).copy_(new)
    kept = (y[row] / new[to][..., None]).clamp(-448.0, 448.0).to(_E4M3)
    cache.view(torch.uint8).flatten(0, 1)[slots[row]] = kept.view(torch.uint8)


def _append_plain(state):
    _store(state, "k", *_turned(state))
    if state["v"] is not None:
        y = state["v"].float()
        _store(state, "v", y, y.abs())


def _slots_of(state, positions):
    """Slots of positions [B, T, n] of each sequence; negative positions stand for slot 0."""
    ps, p = state["case"]["page_size"], positions.clamp(min=0).long()
    pages = torch.gather(state["table"].long(), 1, (p // ps).flatten(1)).view(p.shape)
    return pages * ps + p % ps


def _attention_plain(state):
    case, pos = state["case"], state["indices"]
    B, T, Hq, Hkv = (case[n] for n in ("B", "T", "Hq", "Hkv"))
    slots = _slots_of(state, pos)
    k, v = ((state[n].flatten(0, 1)[slots].float() * state[n + "_scales"].flatten(0, 1)[slots // case["block"]][..., None])
            for n in ("k", "v"))
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
    return out.view(B, T, Hq, -1).to(state["q"].dtype), (torch.log(total) + top).view(B, T, Hq)


# ---- one pass ---------------------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if case["op"] == "append":
        if not own:
            _append_plain(state)
        else:
            import sparse_attention_indexer_fp32_gb300 as tk

            tk.cache_append(state["k"], state["v"], state["positions"], state["frequencies"], state["k_cache"],
                            state["v_cache"], state["slots"], k_scales=state["k_scales"], v_scales=state["v_scales"],
                            layout=case["layout"], offset=case["offset"])
        return {n: state[n] for n in ("k_cache", "k_scales", "v_cache", "v_scales")}
    if not own:
        return _attention_plain(state)
    import sparse_attention_indexer_fp32_gb300 as tk

    return tk.sparse_attention(state["q"], state["k"], state["v"], state["indices"], state["table"],
                               k_scales=state["k_scales"], v_scales=state["v_scales"], query_positions=state["qpos"],
                               scale=state["scale"], softcap=state["cap"], slopes=state["slopes"], first=state["first"],
                               return_lse=True)


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    b = _BYTES[case["type"]]
    if case["op"] == "append":
        T, H, D, Dv, block = case["B"] * case["n"], case["H"], case["D"], case["Dv"], case["block"]
        scales = 0 if not block else case["B"] * -(-case["n"] // block) * H * 4 * (2 if Dv else 1)
        return {"bytes": T * H * (D + Dv) * (b + (1 if block else b)) + scales + 8 * T, "flops": 3 * T * H * case["rotated"]}
    B, T, S, D, Hq, Hkv, Dv, K = (case[n] for n in ("B", "T", "S", "D", "Hq", "Hkv", "Dv", "K"))
    part = 0.5 if case["documents"] else 1.0
    chosen = int(part * B * T * min(K, int(0.9 * S)))
    entries = min(chosen, int(part * 0.9 * B * S))
    entry = Hkv * (D if case["shared"] else D + Dv)
    scales = min(entries, int(0.9 * B * S) // case["block"] + B) * Hkv * (4 if case["shared"] else 8)
    return {"bytes": entries * entry + scales + 4 * B * T * K + B * T * Hq * ((D + Dv) * b + 4),
            "flops": 2 * chosen * Hq * (D + Dv)}


# ---- the definition in 64 bits ----------------------------------------------------------------------


def _exact_side(s, side, y, bound):
    """What one cache and its scales hold afterwards, entries in units of their scale and not rounded again."""
    slots = s["slots"].tolist()
    at = [i for i, slot in enumerate(slots) if slot >= 0]
    to = s["slots"][at].long()
    cache = s[side + "_cache"].double()
    flat = cache.view(-1, *cache.shape[2:])
    if s[side + "_scales"] is None:
        flat[to] = y[at]
        return cache, None
    block, scales = s["case"]["block"], s[side + "_scales"].double()
    rows = scales.view(-1, scales.shape[-1])
    members = {}
    for i in at:
        members.setdefault(slots[i] // block, []).append(i)
    tokens = list(members.values())
    which = torch.tensor(list(members), device=y.device)
    first = torch.tensor([min(slots[i] % block for i in m) for m in tokens], device=y.device)[:, None]
    longest = max(len(m) for m in tokens)
    padded = torch.tensor([m + m[:1] * (longest - len(m)) for m in tokens], device=y.device)
    most = bound[padded].amax(dim=1)
    powers = 2.0 ** torch.arange(-126, 128, dtype=torch.float64)  # the first one that is large enough
    need = powers.to(y.device)[torch.searchsorted(448.0 * powers.to(y.device), most)]
    before = rows[which]
    after = torch.where(first == 0, need, torch.maximum(before, need))
    rows[which] = after
    blocks = flat.view(-1, block, *flat.shape[1:])
    held = torch.arange(block, device=y.device)[None] < first
    blocks[which] = torch.where(held[..., None, None], blocks[which] * (before / after)[:, None, :, None], blocks[which])
    flat[to] = y[at] / rows[to // block][..., None]
    return cache, scales


def _exact_append(s, case):
    k = s["k"].double()
    R, o = case["rotated"], case["offset"]
    turn = s["positions"].double().view(-1, 1, 1) * s["frequencies"].view(1, 1, -1)
    if case["layout"] == "half":
        one, two = slice(o, o + R // 2), slice(o + R // 2, o + R)
    else:
        one, two = slice(o, o + R, 2), slice(o + 1, o + R, 2)
    y, size = k.clone(), k.abs()
    size[..., one] = size[..., two] = size[..., one] + size[..., two]
    z = torch.complex(k[..., one], k[..., two]) * torch.polar(torch.ones_like(turn), turn)
    y[..., one], y[..., two] = z.real, z.imag
    got = {}
    got["k_cache"], got["k_scales"] = _exact_side(s, "k", y, size.amax(dim=-1))
    got["v_cache"] = got["v_scales"] = None
    if s["v"] is not None:
        v = s["v"].double()
        got["v_cache"], got["v_scales"] = _exact_side(s, "v", v, v.abs().amax(dim=-1))
    return got


def _exact_attention(s, case):
    B, T, Hq, Hkv, ps = (case[n] for n in ("B", "T", "Hq", "Hkv", "page_size"))
    out = torch.zeros((B, T, Hq, case["Dv"]), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    head = torch.arange(Hq, device=s["q"].device) // (Hq // Hkv)
    for b in range(B):
        for t0 in range(0, T, 16):
            idx = s["indices"][b, t0:t0 + 16].long()
            safe = idx.clamp(min=0)
            page, place = s["table"][b].long()[safe // ps], safe % ps
            k = s["k"][page, place].double() * s["k_scales"][page, place // case["block"]].double()[..., None]
            v = s["v"][page, place].double() * s["v_scales"][page, place // case["block"]].double()[..., None]
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
    return (_exact_append if case["op"] == "append" else _exact_attention)(s, case)
