"""Cases for the operators around the 4-bit KV cache: the insert with its reader, the
attention over the cache, the attention weights it gathers per key, and the eviction that
goes by them.

Each case runs one operator, either in plain torch operations (``own`` false) or through
the package's entry points (``own`` true), on the same inputs.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD, NOPE, ROPE = 512, 448, 64          # row width, quantised dims, rotated dims
GROUP, GROUPS = 32, 14                   # elements per scale, scales per row
DATA, SCALE = 352, 16                    # bytes per slot: 224 of codes + 128 of bf16, 14 scales + 2
EPS = 1e-6
SOFTMAX_SCALE = HEAD ** -0.5

# Nibble n of a 32-bit word of codes holds element NIBBLE[n] of its eight.
NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of 128 requests: their q heads and new KV rows, a tenth of them padding
        dict(name="insert_decode", op="insert", tokens=128, heads=64, block=64, skip=0.1),
        # KV rows of a long prompt, with the heads left to another device
        dict(name="insert_prefill", op="insert", tokens=100003, heads=0, block=64, skip=0.01),
        # the smallest call: two short requests on few heads, where latency is all
        dict(name="attention_small", op="attention", batch=2, q_len=1, heads=8, low=1, high=130, block=16, window=0, sinks=False),
        # a step of ordinary decoding, ragged lengths with an idle request among them
        dict(name="attention_decode", op="attention", batch=48, q_len=1, heads=64, low=64, high=4096, block=64, window=0, sinks=True),
        # a long document on one request, all heads on this device
        dict(name="attention_long", op="attention", batch=1, q_len=1, heads=128, low=262147, high=262147, block=64, window=0, sinks=False),
        # a full server: many requests of some thousand tokens
        dict(name="attention_large", op="attention", batch=128, q_len=1, heads=128, low=1024, high=8192, block=64, window=0, sinks=False),
        # several drafted tokens verified at once, a sliding window, pages of an odd size
        dict(name="attention_draft", op="attention", batch=24, q_len=3, heads=40, low=1, high=6000, block=27, window=2048, sinks=True),
        # a chunk of a prompt against what is cached before it
        dict(name="attention_chunk", op="attention", batch=2, q_len=160, heads=64, low=2500, high=5001, block=64, window=0, sinks=False),
        # the weights of one decoding step, gathered per key
        dict(name="weights_decode", op="weights", batch=48, q_len=1, heads=64, low=64, high=4096, block=64, window=0),
        # the same over long contexts
        dict(name="weights_long", op="weights", batch=3, q_len=2, heads=128, low=60001, high=131072, block=64, window=0),
        # a batch cut back to a quarter
        dict(name="evict_batch", op="evict", batch=48, low=1500, high=8192, block=64, budget=2048, recent=256),
        # one long request cut to an eighth
        dict(name="evict_long", op="evict", batch=1, low=262144, high=262144, block=64, budget=32768, recent=1000),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["insert", "attention", "attention", "weights", "evict"])
    block = rng.choice([1, 5, 16, 27, 32, 64, 64, 64, 128])
    if op == "insert":
        heads = rng.choice([0, 0, _log(rng, 1, 128)])
        return dict(op=op, tokens=_log(rng, 1, 100003 // (1 + heads)), heads=heads, block=block, skip=rng.choice([0.0, 0.1, 0.5]))
    if op == "evict":
        batch = _log(rng, 1, 64)
        high = _log(rng, 16, min(262144, 400000 // batch))
        budget = _log(rng, 1, high)
        return dict(op=op, batch=batch, low=_log(rng, 1, high), high=high, block=block, budget=budget, recent=rng.randint(0, budget))
    heads, batch = _log(rng, 1, 128), _log(rng, 1, 128)
    q_len = rng.choice([1, 1, rng.randint(2, 6), _log(rng, 1, 200)])
    most = 128 * 128 * 4096 // (heads * batch * q_len)  # pairs of query rows and keys
    most = max(8, min(most, 400000 // batch, 262144))
    high = _log(rng, min(most, 8), most)
    case = dict(op=op, batch=batch, q_len=q_len, heads=heads, low=rng.choice([1, max(1, high // 4), high]), high=high, block=block,
                window=rng.choice([0, 0, _log(rng, 1, high)]))
    if op == "attention":
        case["sinks"] = rng.random() < 0.5
    return case


def lens_of(case):
    """The requests' lengths: ragged between low and high, the last one at high, one of many idle."""
    rng = random.Random("%(batch)d %(low)d %(high)d" % case)
    lens = [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]
    lens[-1] = case["high"]
    if case["batch"] >= 8:
        lens[3] = 0
    return lens


def _pairs(case):
    """(query token, key) pairs that are visible, and the keys that some token sees."""
    pairs = keys = 0
    for n in lens_of(case):
        seen = []
        for j in range(case["q_len"]):
            to = max(0, n - case["q_len"] + 1 + j)
            since = max(0, to - case["window"]) if case["window"] else 0
            pairs += to - since
            seen.append((since, to))
        keys += seen[-1][1] - min(s[0] for s in seen)
    return pairs, keys


def work(case):
    if case["op"] == "insert":
        t, h = case["tokens"], case["heads"]
        # q read and written, kv read, the row written, read back and written out; cos and sin by position
        return {"bytes": t * (h * 2048 + 1024 + 2 * (DATA + SCALE) + 1024 + 256 + 16) + 1024, "flops": t * (h * 3 + 8) * HEAD}
    if case["op"] == "evict":
        lens = lens_of(case)
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 4 * sum(lens) + kept * (2 * (DATA + SCALE) + 4) + 4 * case["budget"] * len(lens), "flops": sum(lens)}
    pairs, keys = _pairs(case)
    rows = case["batch"] * case["q_len"] * case["heads"]
    if case["op"] == "attention":
        return {"bytes": keys * (DATA + SCALE) + rows * (2 * 1024 + 4), "flops": 4 * HEAD * pairs * case["heads"]}
    return {"bytes": keys * (DATA + SCALE + 8) + rows * (1024 + 4), "flops": 2 * HEAD * pairs * case["heads"]}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _pages(case, gen, lens):
    """A cache of shuffled pages: for each request its pages in order, -1 after them."""
    block, wide = case["block"], -(-case["high"] // case["block"])
    pages = [-(-n // block) for n in lens]
    total = sum(pages) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _filled(case, gen, table, total, lens, toward):
    """The cache's bytes: normalised rows of which some lean toward `toward`, in 4 bits; slots past a request's length hold 0xff."""
    block = case["block"]
    cache = torch.empty(total, block * (DATA + SCALE), dtype=torch.uint8, device="cuda")
    step = max(1, 65536 // block)
    for p in range(0, total, step):
        n = min(step, total - p)
        x = torch.randn(n, block, HEAD, generator=gen, device="cuda")
        if toward is not None:
            x += torch.empty(n, block, 1, device="cuda").exponential_(5.0, generator=gen) * toward
        data, scales = encode(_rms(x))
        cache[p:p + n, :block * DATA] = data.reshape(n, -1)
        cache[p:p + n, block * DATA:] = scales.reshape(n, -1)
    stale = torch.ones(total, block, dtype=torch.bool, device="cuda")
    at = torch.arange(table.shape[1] * block, device="cuda")
    live = at < torch.tensor(lens, device="cuda")[:, None]
    slots = (table.long()[:, at // block] * block + at % block)[live]
    stale.view(-1)[slots] = False
    data, scales = _split(cache, block)
    data[stale] = 255
    scales[stale] = 255
    return cache.reshape(-1)


def _split(cache, block):
    pages = cache.view(-1, block * (DATA + SCALE))
    return pages[:, :block * DATA].unflatten(1, (block, DATA)), pages[:, block * DATA:].unflatten(1, (block, SCALE))


def prepare(case, seed):
    gen = _generator(seed)
    s = dict(case)
    if case["op"] == "insert":
        t, h, block = case["tokens"], case["heads"], case["block"]
        blocks = -(-2 * t // block) + 1
        angles = torch.arange(8192, dtype=torch.float64, device="cuda")[:, None] * (
            10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32))
        slots = torch.randperm(blocks * block, generator=gen, device="cuda")[:t]
        skip = torch.rand(t, generator=gen, device="cuda") < case["skip"]
        s.update(
            q=torch.randn(t, h, HEAD, generator=gen, device="cuda").to(torch.bfloat16) if h else None,
            kv=(torch.randn(t, HEAD, generator=gen, device="cuda") *
                (1 + 20 * (torch.rand(t, HEAD, generator=gen, device="cuda") < 0.002))).to(torch.bfloat16),
            weight=(1 + 0.1 * torch.randn(HEAD, generator=gen, device="cuda")).to(torch.bfloat16),
            positions=torch.randint(0, 8192, (t,), generator=gen, device="cuda"),
            cos_sin=torch.cat([angles.cos(), angles.sin()], 1).float(),
            slots=torch.where(skip, -1, slots), blocks=blocks,
            cache=torch.zeros(blocks * block * (DATA + SCALE), dtype=torch.uint8, device="cuda"),
            rows=torch.empty(t, HEAD, dtype=torch.bfloat16, device="cuda"))
        return s
    lens = lens_of(case)
    table, total = _pages(case, gen, lens)
    s.update(table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["op"] == "evict":
        block, batch = case["block"], case["batch"]
        wide = -(-case["budget"] // block)
        cache = _filled(case, gen, table, total, lens, None)
        to = torch.randperm(batch * wide, generator=gen, device="cuda").to(torch.int32).view(batch, wide)
        weights = torch.exp(2 * torch.randn(batch, case["high"], generator=gen, device="cuda"))
        weights[torch.rand(weights.shape, generator=gen, device="cuda") < 0.05] = 0.0  # never attended to
        weights = torch.where(torch.rand(weights.shape, generator=gen, device="cuda") < 0.1, weights.round(), weights)
        s.update(cache=torch.cat([cache, torch.zeros(batch * wide * block * (DATA + SCALE), dtype=torch.uint8, device="cuda")]),
                 blocks=total + batch * wide, first=total, to=to + total, weights=weights,
                 kept=torch.empty(batch, case["budget"], dtype=torch.int32, device="cuda"),
                 new_lens=torch.empty(batch, dtype=torch.int32, device="cuda"),
                 new_weights=torch.empty(batch, case["budget"], device="cuda"))
        return s
    batch, q_len, heads = case["batch"], case["q_len"], case["heads"]
    toward = _rms(torch.randn(HEAD, generator=gen, device="cuda"))
    q = _rms(torch.randn(batch, q_len, heads, HEAD, generator=gen, device="cuda") + 0.5 * toward).to(torch.bfloat16)
    s.update(q=q, cache=_filled(case, gen, table, total, lens, toward), blocks=total,
             lse=torch.empty(batch, q_len, heads, device="cuda"))
    if case["op"] == "attention":
        s.update(out=torch.empty_like(q), sink=torch.randn(heads, generator=gen, device="cuda") if case["sinks"] else None)
    else:
        s["sink"] = None
        s["lse"] = attention(s)[1]
        s["weights"] = torch.zeros(batch, case["high"], device="cuda").exponential_(1.0, generator=gen)
    return s


# ---------------------------------------------------------------- the plain forms

def encode(v):
    """Rows [..., 512] as the cache holds them: (data bytes [..., 352], scale bytes [..., 16])."""
    groups = v[..., :NOPE].unflatten(-1, (GROUPS, GROUP))
    mantissa, exponent = torch.frexp(groups.abs().amax(-1).double())  # amax = mantissa * 2^exponent, mantissa in [1/2, 1)
    s = torch.where(mantissa > 0.75, exponent - 2, exponent - 3).clamp(-127, 127)  # the least s with amax <= 6 * 2^s
    s = torch.where(mantissa == 0, -127, s)
    x = (groups.double() * ((1023 - s.long()) << 52).view(torch.float64)[..., None]).to(v.dtype)
    a = x.abs()
    # the midpoints between neighbouring values; a tie goes to the even code
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.int64)
    code = (code + 8 * (x < 0)).flatten(-2).unflatten(-1, (NOPE // 8, 8))
    word = sum(code[..., e] << (4 * n) for n, e in enumerate(NIBBLE))
    codes = torch.stack([(word >> (8 * i)) & 255 for i in range(4)], -1).flatten(-2).to(torch.uint8)
    tail = v[..., NOPE:].to(torch.bfloat16).contiguous().view(torch.uint8)
    scales = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, SCALE - GROUPS))
    return torch.cat([codes, tail], -1), scales


def decode(data, scales):
    """The fp32 values of rows held as bytes: data [..., 352], scales [..., 16]."""
    low, high = data[..., :224] & 15, data[..., :224] >> 4
    nibbles = torch.stack([low, high], -1).flatten(-2).unflatten(-1, (NOPE // 8, 8))
    order = torch.tensor([NIBBLE.index(e) for e in range(8)], device=data.device)
    codes = nibbles[..., order].flatten(-2)
    values = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=data.device)[codes.int()]
    exponent = scales[..., :GROUPS].int()
    step = torch.where(exponent == 0, 0x00400000, exponent << 23).view(torch.float32)  # 2^(exponent - 127)
    values = (values.unflatten(-1, (GROUPS, GROUP)) * step[..., None]).flatten(-2)
    return torch.cat([values, data[..., 224:].contiguous().view(torch.bfloat16).float()], -1)


def rotate(x, cos_sin):
    """The trailing 64 dims of x turned in neighbouring pairs by the angles of cos_sin [..., 64]."""
    a, b = x[..., NOPE::2], x[..., NOPE + 1::2]
    c, s = cos_sin[..., :32], cos_sin[..., 32:]
    return torch.cat([x[..., :NOPE], torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)], -1)


def insert(s):
    angles = s["cos_sin"][s["positions"]]
    out = {}
    if s["q"] is not None:
        x = s["q"].float()
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        s["q"].copy_(rotate(x, angles[:, None]))
        out["q"] = s["q"]
    # in 64 bits: values next to a border between two codes
    x = s["kv"].double()
    x = rotate(x / (x.square().mean(-1, keepdim=True) + np.float64(np.float32(EPS))).sqrt() * s["weight"].double(), angles.double())
    data, scales = encode(x)
    written = s["slots"] >= 0
    block, at = s["block"], s["slots"][written]
    cache_data, cache_scales = _split(s["cache"], block)
    cache_data[at // block, at % block] = data[written]
    cache_scales[at // block, at % block] = scales[written]
    at = s["slots"].clamp(min=0)
    rows = decode(cache_data[at // block, at % block], cache_scales[at // block, at % block])
    out["rows"] = torch.where(written[:, None], rows, 0.0).to(torch.bfloat16)
    return out


def _scores(s):
    """The scaled scores [B, Q, H, L] of all keys in 32 bits, the mask [B, Q, 1, L] and the keys' rows [B, L, 512]."""
    block = s["block"]
    cache_data, cache_scales = _split(s["cache"], block)
    pages = s["table"].clamp(min=0)
    rows = decode(cache_data[pages], cache_scales[pages]).flatten(1, 2)
    at = torch.arange(rows.shape[1], device="cuda")
    rows = torch.where((at < s["lens"][:, None])[..., None], rows, 0.0)
    q_len = s["q"].shape[1]
    to = (s["lens"][:, None] - q_len + 1 + torch.arange(q_len, device="cuda"))[:, :, None, None]
    seen = at < to
    if s["window"]:
        seen = seen & (at >= to - s["window"])
    scores = torch.matmul(s["q"].float().flatten(1, 2), rows.transpose(1, 2)).unflatten(1, s["q"].shape[1:3])
    return (scores * SOFTMAX_SCALE).masked_fill(~seen, -math.inf), rows


def attention(s):
    scores, rows = _scores(s)
    most = scores.amax(-1, keepdim=True)
    if s["sink"] is not None:
        most = torch.maximum(most, s["sink"][:, None])
    most = torch.where(most == -math.inf, 0.0, most)
    p = torch.exp(scores - most)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][:, None] - most)
    out = torch.matmul(p.flatten(1, 2), rows).unflatten(1, p.shape[1:3])
    out = torch.where(total > 0, out / total, 0.0)
    return out.to(torch.bfloat16), (most + torch.log(total)).squeeze(-1)


def weights(s):
    scores, _ = _scores(s)
    p = torch.exp(scores - torch.where(s["lse"] == -math.inf, 0.0, s["lse"])[..., None])
    s["weights"] += p.sum((1, 2))[:, :s["weights"].shape[1]]
    return s["weights"]


def evict(s):
    lens, budget, block = s["lens"][:, None], s["budget"], s["block"]
    w = torch.where(s["weights"].isnan(), -math.inf, s["weights"])
    at = torch.arange(w.shape[1], device="cuda")
    # by class (the recent, the others, those past the length), then by falling weight, then by index
    kind = torch.where(at < lens - s["recent"], 1, torch.where(at < lens, 0, 2))
    order = torch.sort(w, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(kind.gather(1, order), dim=1, stable=True).indices)[:, :budget]
    new_lens = s["lens"].clamp(max=budget)
    order = torch.nn.functional.pad(order, (0, budget - order.shape[1]))
    live = torch.arange(budget, device="cuda") < new_lens[:, None]
    kept = torch.where(live, order, w.shape[1]).sort(dim=1).values
    new_weights = torch.where(live, s["weights"].gather(1, kept.clamp(max=w.shape[1] - 1)), 0.0)
    kept = torch.where(live, kept, -1).int()
    b, i = torch.nonzero(live, as_tuple=True)
    src, dst = kept[b, i].long(), i
    for part in _split(s["cache"], block):
        part[s["to"].long()[b, dst // block], dst % block] = part[s["table"].long()[b, src // block], src % block]
    return kept, new_lens, new_weights


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        import kv_norm_rope_gb300 as k
    if s["op"] == "insert":
        if not own:
            return insert(s)
        k.qnorm_rope_kv_fp4_insert(s["q"], s["kv"], s["weight"], s["positions"], s["cos_sin"], s["slots"], s["cache"],
                                   s["blocks"], s["block"], EPS)
        k.fp4_dequant_gather(s["cache"], s["blocks"], s["block"], s["slots"], s["rows"])
        return {"rows": s["rows"]} if s["q"] is None else {"q": s["q"], "rows": s["rows"]}
    if s["op"] == "attention":
        if own:
            k.fp4_attention(s["q"], s["cache"], s["blocks"], s["block"], s["table"], s["lens"], SOFTMAX_SCALE, s["out"],
                            lse=s["lse"], sinks=s["sink"], window=s["window"])
            return {"out": s["out"], "lse": s["lse"]}
        out, lse = attention(s)
        return {"out": out, "lse": lse}
    if s["op"] == "weights":
        if own:
            k.fp4_attention_weights(s["q"], s["cache"], s["blocks"], s["block"], s["table"], s["lens"], SOFTMAX_SCALE, s["lse"],
                                    s["weights"], window=s["window"])
            return {"weights": s["weights"]}
        return {"weights": weights(s)}
    if own:
        k.fp4_evict(s["cache"], s["blocks"], s["block"], s["table"], s["lens"], s["weights"], s["budget"], s["recent"], s["to"],
                    s["kept"], s["new_lens"], s["new_weights"])
        kept, new_lens, new_weights = s["kept"], s["new_lens"], s["new_weights"]
    else:
        kept, new_lens, new_weights = evict(s)
    # the rows are moved as bytes: the pages that they were moved to, whole
    moved = s["cache"][s["first"] * s["block"] * (DATA + SCALE):]
    return {"kept": kept, "lens": new_lens, "weights": new_weights, "rows": moved}


# ---------------------------------------------------------------- in 64 bits

def _exact_rows(s, pages):
    """The rows of these pages in float64, one code at a time through a table of the bytes' two values."""
    block = s["block"]
    raw = s["cache"].view(-1, block * (DATA + SCALE))[pages.long()]
    data, scales = raw[:, :block * DATA].reshape(-1, DATA), raw[:, block * DATA:].reshape(-1, SCALE)
    sign_value = [(-1.0 if c & 8 else 1.0) * E2M1[c & 7] for c in range(16)]
    pair = torch.tensor([[sign_value[b & 15], sign_value[b >> 4]] for b in range(256)], dtype=torch.float64, device="cuda")
    out = torch.empty(data.shape[0], HEAD, dtype=torch.float64, device="cuda")
    for i in range(4):  # bytes i of the words: nibbles 2i and 2i + 1
        both = pair[data[:, i:224:4].long()]
        out[:, NIBBLE[2 * i]:NOPE:8], out[:, NIBBLE[2 * i + 1]:NOPE:8] = both[..., 0], both[..., 1]
    out[:, :NOPE] *= torch.pow(2.0, scales[:, :GROUPS].double() - 127).repeat_interleave(GROUP, dim=1)
    out[:, NOPE:] = data[:, 224:].contiguous().view(torch.bfloat16).double()
    return out


def _exact_insert(s):
    out = {}
    turn = torch.complex(*s["cos_sin"].double()[s["positions"]].split(32, dim=1))
    eps = float(np.float32(EPS))

    def turned(x, by):
        z = torch.view_as_complex(x[..., NOPE:].unflatten(-1, (32, 2)).contiguous()) * by
        return torch.cat([x[..., :NOPE], torch.view_as_real(z).flatten(-2)], -1)

    if s["q"] is not None:
        x = s["q"].double()
        out["q"] = turned(x / torch.sqrt((x * x).sum(-1, keepdim=True) / HEAD + eps), turn[:, None])
    x = s["kv"].double()
    x = turned(x / torch.sqrt((x * x).sum(-1, keepdim=True) / HEAD + eps) * s["weight"].double(), turn)
    groups = x[:, :NOPE].reshape(-1, GROUP)
    amax = groups.abs().amax(1, keepdim=True)
    step = torch.full_like(amax, 2.0 ** -127)
    for e in range(-126, 128):  # the least power of two that reaches
        step = torch.where(amax > 6 * step, torch.full_like(step, 2.0 ** e), step)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    at = torch.searchsorted(grid, (groups.abs() / step).contiguous()).clamp(1, 7)
    below, above, y = grid[at - 1], grid[at], groups.abs() / step
    up = (y - below > above - y) | ((y - below == above - y) & (at % 2 == 0))
    x[:, :NOPE] = (torch.where(up, above, below) * step * torch.sign(groups)).reshape(-1, NOPE)
    out["rows"] = torch.where((s["slots"] >= 0)[:, None], x, 0.0)
    return out


def _exact_attention(s):
    q_len, lens = s["q"].shape[1], s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    total = s["weights"].double() if s["op"] == "weights" else None
    for b, n in enumerate(lens):
        rows = _exact_rows(s, s["table"][b][:-(-n // s["block"])])[:n]
        for j in range(q_len):
            to = n - q_len + 1 + j
            since = max(0, to - s["window"]) if s["window"] else 0
            if to <= since:
                if s["sink"] is not None:
                    lse[b, j] = s["sink"].double()
                continue
            x = s["q"][b, j].double() @ rows[since:to].T * SOFTMAX_SCALE
            if total is not None:
                total[b, since:to] += torch.exp(x - s["lse"][b, j].double()[:, None]).sum(0)
                continue
            if s["sink"] is not None:
                x = torch.cat([x, s["sink"].double()[:, None]], 1)
            lse[b, j] = torch.logsumexp(x, 1)
            out[b, j] = torch.softmax(x, 1)[:, :to - since] @ rows[since:to]
    return {"weights": total} if total is not None else {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "evict":
        return None  # nothing is computed: indices and copies
    s = prepare(case, seed)
    return _exact_insert(s) if case["op"] == "insert" else _exact_attention(s)
