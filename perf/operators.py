"""Cases of the 8-bit key/value cache and of the attention steps that read a cache.

Five operators of one decoding loop:

  write      mha_cache_write_f8: new keys and values (bf16) enter an e4m3 cache, one power-of-two scale per position and head
  read       mha_cache_read_f8: cached rows come back as bf16
  decode     mha_decode_f8: one query per sequence over the e4m3 cache
  tree       mha_decode_tree: a tree of drafted tokens per sequence over a bf16 cache
  tree_f8    mha_decode_tree_f8: the same over the e4m3 cache

Layouts: q [B, T, H, d], k and v rows [B, T, H_kv, d], caches [B, Lk, H_kv, d], scales [B, H_kv, Lk] (biased exponents: a byte s stands for
2^(s - 127)), row log-sum-exps [B, H, T] ([B, H] for decode).  H_kv divides H: query head h reads key head h // (H / H_kv).
"""
import math
import random

import torch

own = False

LOWEST_EXPONENT = -64


def listed():
    return [
        # One new token of 32 sentences with 4 beams each enters the base model's cache (the decode step's own shape: latency).
        {"name": "write_base_token", "op": "write", "B": 128, "T": 1, "H_kv": 8, "d": 64, "Lk": 256, "lo": 1, "hi": 1, "packed": True},
        # Four prompts of up to 2048 tokens of the GPT-3-like layer, keys and values read in place from the packed Q|K|V projection.
        {"name": "write_gpt3_prompt", "op": "write", "B": 4, "T": 2048, "H_kv": 96, "d": 128, "Lk": 2100, "lo": 1024, "hi": 2048, "packed": True},
        # The base model's encoder memory of 64 ragged sources comes back as bf16, for a pass that wants plain keys and values.
        {"name": "read_base_memory", "op": "read", "B": 64, "H_kv": 8, "d": 64, "Lk": 512, "lo": 256, "hi": 512},
        # The GPT-3-like cache of four prompts comes back as bf16.
        {"name": "read_gpt3_prompt", "op": "read", "B": 4, "H_kv": 96, "d": 128, "Lk": 2048, "lo": 1024, "hi": 2048},
        # The base model's decode step: 32 sentences x 4 beams, short caches (latency).
        {"name": "decode_base", "op": "decode", "B": 128, "H": 8, "H_kv": 8, "d": 64, "Lk": 256, "lo": 16, "hi": 256},
        # The GPT-3-like decode step: 4 prompts x 4 beams, 96 heads, 2048 context.
        {"name": "decode_gpt3", "op": "decode", "B": 16, "H": 96, "H_kv": 96, "d": 128, "Lk": 2048, "lo": 1024, "hi": 2048},
        # Two long conversations with shared key heads: few rows, the cache split over the whole machine; odd lengths and capacity.
        {"name": "decode_shared_long", "op": "decode", "B": 2, "H": 32, "H_kv": 8, "d": 128, "Lk": 65543, "lo": 40001, "hi": 65537},
        # A dozen drafted tokens per sentence at the base model's sizes (latency).
        {"name": "tree_base", "op": "tree", "B": 32, "T": 12, "H": 8, "H_kv": 8, "d": 64, "Lk": 300, "lo": 30, "hi": 280, "chain": False},
        # A tree of 25 drafted tokens after four GPT-3-like prompts.
        {"name": "tree_gpt3", "op": "tree", "B": 4, "T": 25, "H": 96, "H_kv": 96, "d": 128, "Lk": 2080, "lo": 1024, "hi": 2048, "chain": False},
        # A tree as large as drafting goes, over shared key heads and a long ragged cache.
        {"name": "tree_shared_long", "op": "tree", "B": 3, "T": 63, "H": 32, "H_kv": 8, "d": 128, "Lk": 16411, "lo": 9001, "hi": 16300, "chain": False},
        # The GPT-3-like tree over the 8-bit cache.
        {"name": "tree_f8_gpt3", "op": "tree_f8", "B": 4, "T": 16, "H": 96, "H_kv": 96, "d": 128, "Lk": 2080, "lo": 1024, "hi": 2048, "chain": False},
        # A run of drafted tokens without branches, wide heads, eight queries to a key head, a long 8-bit cache.
        {"name": "tree_f8_wide_chain", "op": "tree_f8", "B": 5, "T": 7, "H": 16, "H_kv": 2, "d": 256, "Lk": 20011, "lo": 7001, "hi": 20000, "chain": True},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "tree", "tree_f8"])
    d = rng.choice([64, 64, 128, 128, 256, 96, 16 * rng.randint(1, 16)])
    H_kv = rng.choice([1, 2, 3, 8, 12, 96, rng.randint(1, 40)])
    B = _log_uniform(rng, 1, 128)
    top = _log_uniform(rng, 1, 65536)
    # at most the largest listed case's cache (two copies of it in 16 bits), and its rows
    while B * H_kv * top * d > 4 * 96 * 2048 * 128:
        B, top = max(1, B // 2), max(1, top * 2 // 3)
    lo = max(1, top // rng.randint(1, 3))
    case = {"op": op, "B": B, "H_kv": H_kv, "d": d, "lo": lo, "hi": top}
    if op == "write":
        T = rng.choice([1, top, rng.randint(1, top)])
        case.update(T=T, lo=max(1, min(lo, T)), hi=T, Lk=top + rng.randint(0, 40), packed=rng.random() < 0.5)
    elif op == "read":
        case.update(Lk=top + rng.randint(0, 40))
    else:
        G = rng.choice([1, 1, 2, 4, 8, rng.randint(1, 8)])
        T = 1 if op == "decode" else rng.choice([2, 5, 16, rng.randint(1, 64)])
        while B * H_kv * top * d * G * T > 3 * 8 * 16300 * 128 * 252:
            T, G = max(1, T // 2), max(1, G // 2)
        case.update(H=H_kv * G, Lk=top + (0 if op == "decode" else T) + rng.randint(0, 40))
        if op != "decode":
            case.update(T=T, chain=rng.random() < 0.3)
    return case


def _lengths(case, rng):
    """B lengths spread evenly over [lo, hi], in an order of the seed's."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]
    rng.shuffle(lens)
    return lens


def _draft_counts(case, rng):
    """One sequence in three drafted fewer tokens than the batch holds."""
    T = case["T"]
    counts = [T if i % 3 else max(1, (2 * T) // 3) for i in range(case["B"])]
    rng.shuffle(counts)
    return counts


def _tree_bits(case, rng):
    """Ancestor bits [B, T, ceil(T / 64)]: bit j of row t is set where drafted token t sees drafted token j (itself and the tokens it follows)."""
    T, words = case["T"], (case["T"] + 63) // 64
    rows = []
    for _ in range(case["B"]):
        seen = []
        for t in range(T):
            parent = -1 if t == 0 or rng.random() < 0.15 else rng.randrange(max(0, t - 6), t)
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << t))
        rows.append([[_signed((s >> (64 * w)) & (2 ** 64 - 1)) for w in range(words)] for s in seen])
    return torch.tensor(rows, dtype=torch.int64)


def _signed(x):
    return x - 2 ** 64 if x >= 2 ** 63 else x


def _randn(shape, gen, std=1.0):
    """bf16 normal values of this shape on the GPU."""
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(std)


def _exponent(amax):
    """The smallest e >= -64 with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    return torch.clamp(x - 9 + (m > 0.875).to(x.dtype), min=LOWEST_EXPONENT)


def _quantise(x):
    """e4m3 codes like x [..., L, H, d] and biased exponents [..., H, L] of rows of values."""
    x = x.float()
    e = _exponent(x.abs().amax(-1))
    codes = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).transpose(-1, -2).contiguous()


def _values(codes, scales, dtype=torch.float32):
    """What codes [B, L, H, d] and biased exponents [B, H, L] stand for."""
    e = scales.transpose(1, 2).to(torch.int32) - 127
    return torch.ldexp(codes.to(dtype), e.unsqueeze(-1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    op, B, H_kv, d, Lk = case["op"], case["B"], case["H_kv"], case["d"], case["Lk"]
    state = {"op": op}
    lens = _lengths(case, rng)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if op == "write":
        T = case["T"]
        if case["packed"]:  # rows of the packed projection: Q | K | V side by side
            qkv = _randn((B, T, 3, H_kv, d), gen)
            state["k"], state["v"] = qkv[:, :, 1], qkv[:, :, 2]
        else:
            state["k"], state["v"] = _randn((B, T, H_kv, d), gen), _randn((B, T, H_kv, d), gen)
        state["start"] = ints([rng.randint(0, Lk - n) for n in lens])
        state["counts"] = ints(lens)
        for n in ("k", "v"):  # what the caches held before
            codes = torch.randint(0, 0x70, (B, Lk, H_kv, d), generator=gen, device="cuda", dtype=torch.uint8)
            state[n + "_cache"] = codes.view(torch.float8_e4m3fn)
            state[n + "_scale"] = torch.randint(110, 130, (B, H_kv, Lk), generator=gen, device="cuda", dtype=torch.uint8)
        return state
    if op == "read":
        state["lens"] = ints(lens)
        for n in ("k", "v"):
            state[n + "_cache"], state[n + "_scale"] = _quantise(_randn((B, Lk, H_kv, d), gen))
            state[n] = torch.zeros((B, Lk, H_kv, d), device="cuda", dtype=torch.bfloat16)
        return state
    T = 1 if op == "decode" else case["T"]
    q = _randn((B, T, case["H"], d), gen)
    state["q"] = q[:, 0].contiguous() if op == "decode" else q
    state["lens"] = ints(lens)
    if op != "decode":
        state["drafts"] = ints(_draft_counts(case, rng))
        state["mask"] = None if case["chain"] else _tree_bits(case, rng).cuda()
    for n in ("k", "v"):
        x = _randn((B, Lk, H_kv, d), gen)
        if op == "tree":
            state[n + "_cache"] = x
        else:
            state[n + "_cache"], state[n + "_scale"] = _quantise(x)
    return state


def _run_own(s):
    from transformer_head_scaled_sdpa_gb300 import binding
    op = s["op"]
    if op == "write":
        binding.mha_cache_write_f8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["start"], counts=s["counts"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "read":
        return binding.mha_cache_read_f8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["lens"], k=s["k"], v=s["v"])
    if op == "decode":
        return binding.mha_decode_f8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["lens"], return_lse=True)
    if op == "tree":
        return binding.mha_decode_tree(s["q"], s["k_cache"], s["v_cache"], s["lens"], draft_lens=s["drafts"], tree_mask=s["mask"], return_lse=True)
    return binding.mha_decode_tree_f8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["lens"], draft_lens=s["drafts"],
                                      tree_mask=s["mask"], return_lse=True)


def _visible(B, T, Lk, lens, drafts, mask):
    """[B, T, Lk]: which cache rows each drafted token sees."""
    dev = lens.device
    pos = torch.arange(Lk, device=dev)
    j = pos[None, :] - lens[:, None]                       # [B, Lk]: the drafted token a row belongs to
    prefix = j < 0
    if drafts is None:                                     # a plain decode step: the prefix alone
        return prefix[:, None, :].expand(B, T, Lk)
    t = torch.arange(T, device=dev)
    in_draft = (j >= 0) & (j < drafts[:, None])
    jc = j.clamp(0, T - 1)
    if mask is None:
        sees = jc[:, None, :] <= t[None, :, None]
    else:
        words = torch.take_along_dim(mask, (jc // 64)[:, None, :].expand(B, T, Lk).long(), dim=2)
        sees = ((words >> (jc % 64)[:, None, :]) & 1) != 0
    live = t[None, :] < drafts[:, None]                    # rows past a sequence's drafts see nothing
    return (prefix[:, None, :] | (in_draft[:, None, :] & sees)) & live[:, :, None]


def _attention(q, k, v, sees):
    """Softmax attention of q [B, T, H, d] over k, v [B, Lk, H_kv, d] where sees [B, T, Lk]: output and log-sum-exp [B, H, T], 32 bits."""
    B, T, H, d = q.shape
    H_kv = k.shape[2]
    G = H // H_kv
    rows = q.float().reshape(B, T, H_kv, G, d).permute(0, 2, 3, 1, 4).reshape(B, H_kv, G * T, d)
    s = torch.matmul(rows, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    s = s.reshape(B, H_kv, G, T, -1).masked_fill_(~sees[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, H_kv, G * T, -1), v.permute(0, 2, 1, 3)).reshape(B, H_kv, G, T, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (torch.where(m == -math.inf, torch.zeros_like(m), m) + total.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, H, d), lse.reshape(B, H, T)


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "write":
        B, T = s["k"].shape[:2]
        Lk = s["k_cache"].shape[1]
        t = torch.arange(Lk, device="cuda")[None, :] - s["start"][:, None]      # the token that lands on a position
        lands = (t >= 0) & (t < s["counts"][:, None])
        t = t.clamp(0, T - 1).long()
        b = torch.arange(B, device="cuda")[:, None]
        for n in ("k", "v"):
            codes, scales = _quantise(s[n])
            old = s[n + "_cache"].view(torch.uint8)
            old.copy_(torch.where(lands[:, :, None, None], codes.view(torch.uint8)[b, t], old))
            new = torch.take_along_dim(scales, t[:, None, :].expand(-1, scales.shape[1], -1), dim=2)
            s[n + "_scale"].copy_(torch.where(lands[:, None, :], new, s[n + "_scale"]))
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "read":
        Lk = s["k"].shape[1]
        held = (torch.arange(Lk, device="cuda")[None, :] < s["lens"][:, None])[:, :, None, None]
        for n in ("k", "v"):
            s[n].copy_(torch.where(held, _values(s[n + "_cache"], s[n + "_scale"]).to(torch.bfloat16), s[n]))
        return s["k"], s["v"]
    q = s["q"].unsqueeze(1) if op == "decode" else s["q"]
    B, T = q.shape[:2]
    Lk = s["k_cache"].shape[1]
    if op == "tree":
        k, v = s["k_cache"].float(), s["v_cache"].float()
    else:
        k, v = _values(s["k_cache"], s["k_scale"]), _values(s["v_cache"], s["v_scale"])
    o, lse = _attention(q, k, v, _visible(B, T, Lk, s["lens"], s.get("drafts"), s.get("mask")))
    o = o.to(torch.bfloat16)
    return (o[:, 0], lse[:, :, 0]) if op == "decode" else (o, lse)


def exact(case, seed):
    """From the definitions, one sequence and one key head at a time, in float64."""
    s = prepare(case, seed)
    op, B, H_kv, d = case["op"], case["B"], case["H_kv"], case["d"]
    if B * H_kv > 20000:
        return None
    if op == "write":
        out = []
        for n in ("k", "v"):
            cache = s[n + "_cache"].to(torch.float64)
            for b, (at, count) in enumerate(zip(s["start"].tolist(), s["counts"].tolist())):
                x = s[n][b, :count].double()
                top = x.abs().amax(-1, keepdim=True)
                e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0))
                # log2 may round across an integer: settle it on the numbers themselves
                e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
                e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp_min(LOWEST_EXPONENT)
                y = x / torch.exp2(e)
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
                cache[b, at:at + count] = torch.round(y / step) * step
            out.append(cache)
        return out[0], out[1], None, None
    if op == "read":
        out = []
        for n in ("k", "v"):
            x = s[n].double()
            for b, count in enumerate(s["lens"].tolist()):
                e = s[n + "_scale"][b, :, :count].double().t() - 127.0
                x[b, :count] = s[n + "_cache"][b, :count].to(torch.float64) * torch.exp2(e)[:, :, None]
            out.append(x)
        return tuple(out)
    q = s["q"][:, None] if op == "decode" else s["q"]
    T, H, Lk = q.shape[1], case["H"], case["Lk"]
    G = H // H_kv
    o = torch.zeros((B, T, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    bits = s["mask"].cpu().tolist() if s.get("mask") is not None else None
    for b, n in enumerate(s["lens"].tolist()):
        live = T if op == "decode" else int(s["drafts"][b])
        end = n if op == "decode" else min(Lk, n + live)
        hidden = torch.zeros((live, end), dtype=torch.bool)
        for t in range(live):
            for j in range(end - n):
                row = bits[b][t][j // 64] if bits is not None else None
                hidden[t, n + j] = (j > t) if row is None else not (row >> (j % 64)) & 1
        hidden = hidden.cuda()
        for h in range(H_kv):
            kv = []
            for c in ("k", "v"):
                x = s[c + "_cache"][b, :end, h].to(torch.float64)
                if op != "tree":
                    x = x * torch.exp2(s[c + "_scale"][b, h, :end].double() - 127.0)[:, None]
                kv.append(x)
            qs = q[b, :live, h * G:(h + 1) * G].double()                      # [live, G, d]
            a = torch.einsum("tgd,nd->tgn", qs, kv[0]) / math.sqrt(d)
            a = a.masked_fill(hidden[:, None, :], -math.inf)
            z = torch.logsumexp(a, -1)
            o[b, :live, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.exp(a - z[..., None]), kv[1])
            lse[b, h * G:(h + 1) * G, :live] = z.t()
    return (o[:, 0], lse[:, :, 0]) if op == "decode" else (o, lse)


def work(case):
    op, B, H_kv, d = case["op"], case["B"], case["H_kv"], case["d"]
    keys = sum(_lengths(case, random.Random(0)))
    codes = 2 * keys * H_kv * (d + 1)              # keys and values in 8 bits with their exponents
    plain = 2 * keys * H_kv * d * 2                # the same in bf16
    if op in ("write", "read"):
        return {"bytes": codes + plain + 4 * B * (2 if op == "write" else 1), "flops": 2.0 * 2 * keys * H_kv * d}
    H = case["H"]
    if op == "decode":
        rows, drafted, pairs = B, 0, float(keys)
    else:
        counts = _draft_counts(case, random.Random(0))
        rows, drafted = B * case["T"], sum(counts)
        # every live row sees its sequence's prefix; of the drafted tokens, itself at least
        pairs = keys / B * drafted + drafted
        codes += 2 * drafted * H_kv * (d + 1)
        plain += 2 * drafted * H_kv * d * 2
    cache = plain if op == "tree" else codes
    return {"bytes": cache + rows * H * (4 * d + 4) + 4 * B, "flops": 4.0 * d * H * pairs}
