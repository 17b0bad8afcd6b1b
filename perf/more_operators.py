"""Cases of the 4-bit key/value cache, of the attention steps that read it, and of moving cached rows.

Operators of one decoding loop:

  store      mha_cache_write_q4, then mha_cache_read_q4: new keys and values (bf16) enter the 4-bit cache, and the cache comes back as bf16
             (what a prompt's own attention reads, so that it sees the keys that later steps will see)
  decode     mha_decode_q4: one query per sequence over the 4-bit cache
  tree       mha_decode_tree_q4: a tree of drafted tokens per sequence over the 4-bit cache
  fork       mha_cache_fork: beams that did not survive take over the cached rows of those that did
  compact    mha_cache_compact: the accepted drafted tokens' rows move to the end of the prefix

The 4-bit format: a row x of d values (a position and head) has an offset lo = min x and a step, the smallest bf16 number that is at least
(max x - lo) / 15, 2^-13 max |x| and 2^-60; code c is the integer nearest to (x - lo) / step (a tie: the lower) and stands for lo + c step.

Layouts: q [B, T, H, d], k and v rows [B, T, H_kv, d], codes [B, Lk, H_kv, d / 2] (feature 2 i in the low four bits of byte i, 2 i + 1 in the
high ones), (lo, step) bf16 [B, H_kv, Lk, 2], row log-sum-exps [B, H, T] ([B, H] for decode).  H_kv divides H: query head h reads key head
h // (H / H_kv).  Rows are moved in bf16 caches [B, Lk, H_kv, d] and in e4m3 ones with their exponents [B, H_kv, Lk].
"""
import math
import random

import torch

own = False

LEAST_STEP = 2.0 ** -60


def listed():
    return [
        # The base model's encoder memory of 64 ragged sources enters its cache and comes back.
        {"name": "store_base_memory", "op": "store", "B": 64, "T": 512, "H_kv": 8, "d": 64, "Lk": 512, "lo": 256, "hi": 512, "packed": True},
        # A chunk of four GPT-3-like prompts enters behind what is cached, and all of it comes back for the chunk's attention.
        {"name": "store_gpt3_chunk", "op": "store", "B": 4, "T": 512, "H_kv": 96, "d": 128, "Lk": 2085, "lo": 300, "hi": 512, "packed": True},
        # The base model's decode step: 32 sentences x 4 beams, short caches (latency).
        {"name": "decode_base", "op": "decode", "B": 128, "H": 8, "H_kv": 8, "d": 64, "Lk": 256, "lo": 16, "hi": 256},
        # The GPT-3-like decode step: 4 prompts x 4 beams, 96 heads, 2048 context.
        {"name": "decode_gpt3", "op": "decode", "B": 16, "H": 96, "H_kv": 96, "d": 128, "Lk": 2048, "lo": 1024, "hi": 2048},
        # Two long conversations with shared key heads: few rows, the cache split over the whole machine; odd lengths and capacity.
        {"name": "decode_shared_long", "op": "decode", "B": 2, "H": 32, "H_kv": 8, "d": 128, "Lk": 65543, "lo": 40001, "hi": 65537},
        # A dozen drafted tokens per sentence at the base model's sizes (latency).
        {"name": "tree_base", "op": "tree", "B": 32, "T": 12, "H": 8, "H_kv": 8, "d": 64, "Lk": 300, "lo": 30, "hi": 280, "chain": False},
        # A tree of 16 drafted tokens after four GPT-3-like prompts.
        {"name": "tree_gpt3", "op": "tree", "B": 4, "T": 16, "H": 96, "H_kv": 96, "d": 128, "Lk": 2080, "lo": 1024, "hi": 2048, "chain": False},
        # A run of drafted tokens without branches, wide heads, eight queries to a key head, a long cache.
        {"name": "tree_wide_chain", "op": "tree", "B": 5, "T": 7, "H": 16, "H_kv": 2, "d": 256, "Lk": 20011, "lo": 7001, "hi": 20000, "chain": True},
        # 32 sentences x 4 beams of the base model after a beam step, bf16 (latency).
        {"name": "fork_base", "op": "fork", "B": 128, "H_kv": 8, "d": 64, "Lk": 256, "lo": 16, "hi": 256, "f8": False},
        # 4 GPT-3-like prompts x 4 beams, 8-bit: what was generated since the prompt forks.
        {"name": "fork_gpt3", "op": "fork", "B": 16, "H_kv": 96, "d": 128, "Lk": 2048, "lo": 1024, "hi": 2048, "f8": True},
        # The accepted tokens of 32 base model trees, 8-bit (latency).
        {"name": "compact_base", "op": "compact", "B": 32, "T": 12, "H_kv": 8, "d": 64, "Lk": 300, "lo": 30, "hi": 280, "f8": True},
        # The accepted tokens of trees of 63 over four GPT-3-like prompts, bf16.
        {"name": "compact_gpt3", "op": "compact", "B": 4, "T": 63, "H_kv": 96, "d": 128, "Lk": 2113, "lo": 1024, "hi": 2048, "f8": False},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "decode", "tree", "decode", "tree", "fork", "compact"])
    d = rng.choice([64, 64, 128, 128, 256, 96, 32 * rng.randint(1, 8)])
    H_kv = rng.choice([1, 2, 3, 8, 12, 96, rng.randint(1, 40)])
    B = _log_uniform(rng, 1, 128)
    top = _log_uniform(rng, 1, 65536)
    # at most the largest listed cases' bytes
    while B * H_kv * top * d > {"store": 1, "fork": 3}.get(op, 12) * 96 * 2048 * 128:
        B, top = max(1, B // 2), max(1, top * 2 // 3)
    lo = max(1, top // rng.randint(1, 3))
    case = {"op": op, "B": B, "H_kv": H_kv, "d": d, "lo": lo, "hi": top}
    if op == "store":
        T = rng.choice([1, top, rng.randint(1, top)])
        case.update(T=T, lo=max(1, min(lo, T)), hi=T, Lk=top + rng.randint(0, 40), packed=rng.random() < 0.5)
    elif op == "fork":
        case.update(Lk=top + rng.randint(0, 40), f8=rng.random() < 0.5)
    elif op == "compact":
        T = rng.randint(2, 64)
        case.update(T=T, Lk=top + T + rng.randint(0, 40), f8=rng.random() < 0.5)
    else:
        G = rng.choice([1, 1, 2, 4, 8, rng.randint(1, 8)])
        T = 1 if op == "decode" else rng.choice([2, 5, 16, rng.randint(1, 64)])
        while B * H_kv * top * d * G * T > 5 * 2 * 20000 * 256 * 56:
            T, G = max(1, T // 2), max(1, G // 2)
            if T * G == 1:
                break
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


def _parents(case, rng):
    """The sequence whose rows each one goes on with: in every group of four beams one to three survive and stay where they are."""
    parents = []
    for g in range(0, case["B"], 4):
        group = list(range(g, min(g + 4, case["B"])))
        alive = rng.sample(group, rng.randint(1, max(1, len(group) - 1)))
        parents += [b if b in alive else rng.choice(alive) for b in group]
    return parents


def _paths(case, rng):
    """Accepted drafted tokens, root first, and their numbers: tokens are numbered level by level, so a path either follows the first ones or
    soon has numbers past its own length."""
    T = case["T"]
    rows, counts = [], []
    for _ in range(case["B"]):
        n = rng.randint(1, max(1, min(T, 2 + T // 5)))
        kept = rng.randint(0, n)
        later = sorted(rng.sample(range(n, T), min(n - kept, T - n)))
        path = list(range(kept)) + later
        counts.append(len(path))
        rows.append(path + [0] * (T - len(path)))
    return rows, counts


def _randn(shape, gen, std=1.0):
    """bf16 normal values of this shape on the GPU."""
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(std)


def _step(spread, amax):
    """The smallest bf16 number that is at least spread / 15, 2^-13 amax and 2^-60 (64-bit inputs, exact; 32-bit result)."""
    least = torch.maximum(spread / torch.full_like(spread, 15.0), (amax * 2.0 ** -13).clamp_min(LEAST_STEP))
    near = least.float()
    below = near.double() < least
    bits = near.view(torch.int32) + below.to(torch.int32)
    return (((bits + 0xFFFF) >> 16) << 16).view(torch.float32)


def _quantise(x):
    """Packed codes [..., L, H, d / 2] and (lo, step) [..., H, L, 2] of rows [..., L, H, d] of values."""
    x = x.double()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    step = _step(hi - lo, torch.maximum(hi.abs(), lo.abs()))
    c = torch.ceil((x - lo) / step.double() - 0.5).to(torch.uint8)
    scales = torch.cat((lo.float(), step), -1).to(torch.bfloat16)
    return c[..., 0::2] | (c[..., 1::2] << 4), scales.transpose(-2, -3).contiguous()


def _values(codes, scales, dtype=torch.float32):
    """What packed codes [B, L, H, d / 2] and (lo, step) [B, H, L, 2] stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    s = scales.transpose(1, 2).to(dtype)
    return c.to(dtype) * s[..., 1:] + s[..., :1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    op, B, H_kv, d, Lk = case["op"], case["B"], case["H_kv"], case["d"], case["Lk"]
    state = {"op": op}
    lens = _lengths(case, rng)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if op == "store":
        T = case["T"]
        if case["packed"]:  # rows of the packed projection: Q | K | V side by side
            qkv = _randn((B, T, 3, H_kv, d), gen)
            state["k_new"], state["v_new"] = qkv[:, :, 1], qkv[:, :, 2]
        else:
            state["k_new"], state["v_new"] = _randn((B, T, H_kv, d), gen), _randn((B, T, H_kv, d), gen)
        start = [rng.randint(0, Lk - n) for n in lens]
        state["start"], state["counts"], state["lens"] = ints(start), ints(lens), ints([a + n for a, n in zip(start, lens)])
        for n in ("k", "v"):  # what the caches held before, and where the rows come back to
            state[n + "_cache"], state[n + "_scale"] = _quantise_by_sequence(_randn((B, Lk, H_kv, d), gen))
            state[n] = torch.zeros((B, Lk, H_kv, d), device="cuda", dtype=torch.bfloat16)
        return state
    state["lens"] = ints(lens)
    if op in ("fork", "compact"):
        for n in ("k", "v"):
            x = _randn((B, Lk, H_kv, d), gen)
            state[n + "_cache"] = x.to(torch.float8_e4m3fn) if case["f8"] else x
            if case["f8"]:
                state[n + "_scale"] = torch.randint(110, 130, (B, H_kv, Lk), generator=gen, device="cuda", dtype=torch.uint8)
        if op == "fork":
            state["parent"] = ints(_parents(case, rng))
            state["first"] = ints([rng.randint(0, n) for n in lens])  # what came before is the same in all beams
        else:
            path, counts = _paths(case, rng)
            state["path"], state["counts"] = ints(path), ints(counts)
        return state
    T = 1 if op == "decode" else case["T"]
    q = _randn((B, T, case["H"], d), gen)
    state["q"] = q[:, 0].contiguous() if op == "decode" else q
    if op == "tree":
        state["drafts"] = ints(_draft_counts(case, rng))
        state["mask"] = None if case["chain"] else _tree_bits(case, rng).cuda()
    for n in ("k", "v"):
        state[n + "_cache"], state[n + "_scale"] = _quantise_by_sequence(_randn((B, Lk, H_kv, d), gen))
    return state


def _quantise_by_sequence(x):
    parts = [_quantise(row[None]) for row in x]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _run_own(s):
    from transformer_head_scaled_sdpa_gb300 import binding
    op = s["op"]
    cache = (s["k_cache"], s["v_cache"])
    if op in ("fork", "compact"):
        scales = {"k_scale": s.get("k_scale"), "v_scale": s.get("v_scale")}
        if op == "fork":
            binding.mha_cache_fork(*cache, s["parent"], s["lens"], first=s["first"], **scales)
        else:
            binding.mha_cache_compact(*cache, s["lens"], s["path"], path_lens=s["counts"], **scales)
        return [s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in s]
    cache += (s["k_scale"], s["v_scale"])
    if op == "store":
        binding.mha_cache_write_q4(s["k_new"], s["v_new"], *cache, s["start"], counts=s["counts"])
        return (*binding.mha_cache_read_q4(*cache, s["lens"], k=s["k"], v=s["v"]), s["k_scale"], s["v_scale"])
    if op == "decode":
        return binding.mha_decode_q4(s["q"], *cache, s["lens"], return_lse=True)
    return binding.mha_decode_tree_q4(s["q"], *cache, s["lens"], draft_lens=s["drafts"], tree_mask=s["mask"], return_lse=True)


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


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    B, Lk = s["k_cache"].shape[:2]
    pos = torch.arange(Lk, device="cuda")[None, :]
    if op == "store":
        T = s["k_new"].shape[1]
        t = pos - s["start"][:, None]                       # the token that lands on a position
        lands = (t >= 0) & (t < s["counts"][:, None])
        t = t.clamp(0, T - 1).long()
        b = torch.arange(B, device="cuda")[:, None]
        held = (pos < s["lens"][:, None])[:, :, None, None]
        for n in ("k", "v"):
            codes, scales = _quantise(s[n + "_new"])
            s[n + "_cache"].copy_(torch.where(lands[:, :, None, None], codes[b, t], s[n + "_cache"]))
            new = torch.take_along_dim(scales, t[:, None, :, None].expand(-1, scales.shape[1], -1, 2), dim=2)
            s[n + "_scale"].copy_(torch.where(lands[:, None, :, None], new, s[n + "_scale"]))
            s[n].copy_(torch.where(held, _values(s[n + "_cache"], s[n + "_scale"]).to(torch.bfloat16), s[n]))
        return s["k"], s["v"], s["k_scale"], s["v_scale"]
    if op == "fork":
        moves = (pos >= s["first"][:, None]) & (pos < s["lens"][:, None])
        parent = s["parent"].long()
        for n in ("k", "v"):
            c = _bytes(s[n + "_cache"])
            c.copy_(torch.where(moves[:, :, None, None], c[parent], c))
            if n + "_scale" in s:
                e = s[n + "_scale"]
                e.copy_(torch.where(moves[:, None, :], e[parent], e))
        return [s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in s]
    if op == "compact":
        i = pos[:, :s["path"].shape[1]]
        to = (s["lens"][:, None] + i).long()
        source = torch.where(i < s["counts"][:, None], s["lens"][:, None] + s["path"], to).long()
        b = torch.arange(B, device="cuda")[:, None]
        for n in ("k", "v"):
            c = _bytes(s[n + "_cache"])
            c[b, to] = c[b, source]
            if n + "_scale" in s:
                e = s[n + "_scale"].transpose(1, 2)
                e[b, to] = e[b, source]
        return [s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in s]
    q = s["q"].unsqueeze(1) if op == "decode" else s["q"]
    T = q.shape[1]
    k, v = _values(s["k_cache"], s["k_scale"]), _values(s["v_cache"], s["v_scale"])
    o, lse = _attention(q, k, v, _visible(B, T, Lk, s["lens"], s.get("drafts"), s.get("mask")))
    o = o.to(torch.bfloat16)
    return (o[:, 0], lse[:, :, 0]) if op == "decode" else (o, lse)


def _exact_rows(x):
    """float64 values that rows [..., d] of values stand for once they are cached, and their (lo, step)."""
    x = x.double()
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    fifteen = torch.full_like(lo, 15.0)                     # (a division by a plain number multiplies by its reciprocal)
    least = torch.maximum((hi - lo) / fifteen, x.abs().max(-1, keepdim=True).values / 8192.0).clamp_min(LEAST_STEP)
    m, e = torch.frexp(least)                               # 8 significant bits, rounded up; exact as a bf16 number
    step = torch.ldexp(torch.ceil(m * 256.0), e - 8).to(torch.bfloat16).double()
    at = (x - lo) / step
    c = torch.floor(at)
    return lo + (c + (at - c > 0.5)) * step, torch.cat((lo, step), -1)


def exact(case, seed):
    """From the definitions, one sequence and one key head at a time, in float64."""
    s = prepare(case, seed)
    op, B, H_kv, d = case["op"], case["B"], case["H_kv"], case["d"]
    if op in ("fork", "compact") or B * H_kv > 20000:
        return None
    if op == "store":
        out, scales = [], []
        for n in ("k", "v"):
            rows, pairs = s[n].double(), s[n + "_scale"].double()
            for b, (at, count, held) in enumerate(zip(s["start"].tolist(), s["counts"].tolist(), s["lens"].tolist())):
                c = s[n + "_cache"][b, :held].long()
                c = torch.stack((c % 16, c // 16), -1).reshape(held, H_kv, d).double()
                rows[b, :held] = pairs[b, :, :held, 0].t()[:, :, None] + c * pairs[b, :, :held, 1].t()[:, :, None]
                rows[b, at:at + count], new = _exact_rows(s[n + "_new"][b, :count])
                pairs[b, :, at:at + count] = new.transpose(0, 1)
            out.append(rows)
            scales.append(pairs)
        return (*out, *scales)
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
                x = s[c + "_cache"][b, :end, h].long()
                x = torch.stack((x % 16, x // 16), -1).reshape(end, d).double()
                pair = s[c + "_scale"][b, h, :end].double()
                kv.append(pair[:, :1] + x * pair[:, 1:])
            qs = q[b, :live, h * G:(h + 1) * G].double()                      # [live, G, d]
            a = torch.einsum("tgd,nd->tgn", qs, kv[0]) / math.sqrt(d)
            a = a.masked_fill(hidden[:, None, :], -math.inf)
            z = torch.logsumexp(a, -1)
            o[b, :live, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.exp(a - z[..., None]), kv[1])
            lse[b, h * G:(h + 1) * G, :live] = z.t()
    return (o[:, 0], lse[:, :, 0]) if op == "decode" else (o, lse)


def work(case):
    op, B, H_kv, d = case["op"], case["B"], case["H_kv"], case["d"]
    rng = random.Random(0)
    lens = _lengths(case, rng)
    keys = sum(lens)
    row = d // 2 + 4                               # a key's (or value's) codes with its offset and step
    if op == "store":
        held = keys + sum(rng.randint(0, case["Lk"] - n) for n in lens)
        # new rows in, their codes out, what was cached before read, everything out as bf16
        return {"bytes": 2 * H_kv * (keys * (2 * d + row) + (held - keys) * row + held * 2 * d) + 12 * B, "flops": 2.0 * 2 * (keys + held) * H_kv * d}
    if op in ("fork", "compact"):
        row = H_kv * (d + 1 if case["f8"] else 2 * d)
        if op == "fork":
            parents = _parents(case, rng)
            first = [rng.randint(0, n) for n in lens]
            moved = [(p, n - f) for b, (p, f, n) in enumerate(zip(parents, first, lens)) if p != b]
            most = {}
            for p, n in moved:
                most[p] = max(most.get(p, 0), n)
            rows = sum(n for _, n in moved) + sum(most.values())
        else:
            path, counts = _paths(case, rng)
            rows = 2 * sum(sum(p[i] != i for i in range(n)) for p, n in zip(path, counts))
        return {"bytes": 2 * rows * row + 12 * B, "flops": 0.0}
    H = case["H"]
    if op == "decode":
        rows, drafted, pairs = B, 0, float(keys)
    else:
        counts = _draft_counts(case, random.Random(0))
        rows, drafted = B * case["T"], sum(counts)
        # every live row sees its sequence's prefix; of the drafted tokens, itself at least
        pairs = keys / B * drafted + drafted
    return {"bytes": 2 * (keys + drafted) * H_kv * row + rows * H * (4 * d + 4) + 4 * B, "flops": 4.0 * d * H * pairs}
