"""Cases for the operators around decoding with drafted tokens: the attention over the FP8 and
bf16 KV caches, for chains of new tokens and for trees of drafted ones, the move that keeps the
accepted path's rows, the table of rotary angles, and the rotation of rows by it.

Each case runs one operator, either in plain torch operations (``own`` false) or through
the package's entry points (``own`` true), on the same inputs.
"""
import math
import random

import torch

own = False

HEAD, NOPE, ROPE = 512, 448, 64              # row width, quantised dims, rotated dims
GROUP, GROUPS = 64, 7                        # elements per scale of the FP8 cache, scales a row
# bytes of a slot: a data row, and a scale row after a block's data rows
SLOT = {"fp8": (576, 8), "bf16": (1024, 0), "fp4": (352, 16), "indexer": (128, 4)}
SOFTMAX_SCALE = HEAD ** -0.5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the smallest call: two short requests on few heads, where latency is all
        dict(name="attention_small", op="attention", store="fp8", batch=2, q_len=1, heads=8, low=1, high=130, block=16, window=0, sinks=False),
        # a step of ordinary decoding, ragged lengths with an idle request among them
        dict(name="attention_decode", op="attention", store="fp8", batch=48, q_len=1, heads=64, low=64, high=4096, block=64, window=0, sinks=True),
        # a long document on one request, all heads on this device, rows in bf16
        dict(name="attention_long", op="attention", store="bf16", batch=1, q_len=1, heads=128, low=262147, high=262147, block=64, window=0, sinks=False),
        # a full server: many requests of some thousand tokens
        dict(name="attention_large", op="attention", store="fp8", batch=128, q_len=1, heads=128, low=1024, high=8192, block=64, window=0, sinks=False),
        # a server that verifies a small tree for each request at once; some drafted fewer
        dict(name="tree_verify", op="tree", store="fp8", batch=32, q_len=16, heads=64, low=64, high=4096, block=64, window=0, sinks=False),
        # wide trees of an odd size on few requests, a sliding window, pages of an odd size
        dict(name="tree_wide", op="tree", store="bf16", batch=6, q_len=61, heads=128, low=61, high=8191, block=27, window=4096, sinks=True),
        # after the verification of such a batch: the accepted rows move together
        dict(name="keep_batch", op="keep", store="fp8", batch=32, q_len=16, low=64, high=4096, block=64),
        # the most drafted tokens on many short requests, rows in bf16
        dict(name="keep_wide", op="keep", store="bf16", batch=256, q_len=64, low=64, high=300, block=32),
        # the whole table for a context stretched to a million positions
        dict(name="table_long", op="table", count=1048576, dim=64, scaling="yarn", factor=16.0, given=False),
        # only the rows that a step needs, of far positions
        dict(name="table_step", op="table", count=4099, dim=64, scaling="ntk", factor=8.0, given=True),
        # a decoding step's attention output turned back in place
        dict(name="rows_decode", op="rows", tokens=128, heads=64, width=512, offset=448, dim=64, type="bf16", layout="pairs", inverse=True, inplace=True),
        # a prompt's keys turned out of place, half layout, the first half of the head
        dict(name="rows_prefill", op="rows", tokens=16383, heads=32, width=128, offset=0, dim=64, type="fp16", layout="half", inverse=False, inplace=False),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "tree", "tree", "keep", "table", "rows"])
    block = rng.choice([1, 5, 16, 27, 32, 64, 64, 64, 128])
    if op == "table":
        dim = 2 * _log(rng, 1, 128)
        return dict(op=op, count=_log(rng, 1, 1048576 * 64 // max(dim, 64)), dim=dim, scaling=rng.choice(["plain", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 8.0, 40.0]), given=rng.random() < 0.5)
    if op == "rows":
        width = rng.choice([64, 96, 128, 192, 512, 2 * _log(rng, 1, 300)])
        dim = min(256, rng.choice([width, width // 4 * 2, 2 * rng.randint(1, width // 2)]))
        dim = max(2, dim)
        heads, kind = _log(rng, 1, 128), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        token = heads * width * (8 if kind == "fp32" else 4) + 4 * dim + 8  # bytes
        return dict(op=op, tokens=_log(rng, 1, max(1, 270000000 // token)), heads=heads, width=width,
                    offset=rng.choice([0, width - dim, rng.randint(0, width - dim)]), dim=dim, type=kind,
                    layout=rng.choice(["pairs", "half"]), inverse=rng.random() < 0.5, inplace=rng.random() < 0.5)
    batch = _log(rng, 1, 128)
    if op == "keep":
        q_len = rng.randint(1, 64)
        high = _log(rng, q_len, 4096)
        return dict(op=op, store=rng.choice(sorted(SLOT)), batch=batch, q_len=q_len, low=q_len, high=high, block=block)
    heads = _log(rng, 1, 128)
    q_len = rng.choice([1, 1, rng.randint(2, 6), _log(rng, 1, 200)]) if op == "attention" else _log(rng, 2, 64)
    q_len = max(1, min(q_len, 45000 // (heads * batch)))
    most = 128 * 128 * 4096 // (heads * batch * q_len)  # pairs of query rows and keys
    most = max(8, min(most, 250000 // batch))
    high = _log(rng, min(most, 8), most)
    window = rng.choice([0, 0, _log(rng, 1, high)])
    if op == "tree" and window:
        window = max(window, q_len)
    return dict(op=op, store=rng.choice(["fp8", "bf16"]), batch=batch, q_len=q_len, heads=heads, low=rng.choice([1, max(1, high // 4), high]),
                high=high, block=block, window=window, sinks=rng.random() < 0.5)


def lens_of(case):
    """The requests' lengths: ragged between low and high, the last one at high, one of many idle."""
    rng = random.Random("%(batch)d %(low)d %(high)d" % case)
    lens = [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]
    lens[-1] = case["high"]
    if case["batch"] >= 8:
        lens[3] = 0
    return lens


def trees_of(case):
    """For each request its drafted tokens' ancestors and themselves as bits; 0 for tokens that it did not draft."""
    rng = random.Random("%(batch)d %(q_len)d" % case)
    trees = []
    for b in range(case["batch"]):
        drafted = case["q_len"] if b % 3 else max(1, case["q_len"] - rng.randint(0, case["q_len"] // 2))
        bits = []
        for j in range(drafted):
            # a root, then children of one of the latest tokens
            parent = rng.randint(max(0, j - 6), j - 1) if j else None
            bits.append((1 << j) | (bits[parent] if j else 0))
        trees.append(bits + [0] * (case["q_len"] - drafted))
    return trees


def paths_of(case):
    """For each request the drafted tokens that were accepted, in rising order."""
    rng = random.Random("%(batch)d %(q_len)d %(high)d" % case)
    return [sorted(rng.sample(range(case["q_len"]), rng.randint(0, case["q_len"]) if n else 0)) for n in lens_of(case)]


def _pairs(case):
    """(query token, key) pairs that are visible, and the keys that some token sees."""
    pairs = keys = 0
    trees = trees_of(case) if case["op"] == "tree" else None
    for b, n in enumerate(lens_of(case)):
        c = n - case["q_len"]
        start, drafted = max(c, 0), 0
        for j in range(case["q_len"]):
            if trees is None:
                to, own_keys = max(0, c + 1 + j), 0
                since = max(0, to - case["window"]) if case["window"] else 0
                drafted, start = max(drafted, to), min(start, since)
            else:
                bits = trees[b][j] >> max(0, -c) if n else 0
                own_keys = bin(bits).count("1")
                to = max(c, 0) if trees[b][j] else 0
                since = min(to, max(0, c + bin(trees[b][j]).count("1") - case["window"])) if case["window"] else 0
                if trees[b][j] and n:
                    start, drafted = min(start, since), drafted | bits
            pairs += to - since + own_keys
        keys += drafted - min(start, drafted) if trees is None else max(c, 0) - start + bin(drafted).count("1")
    return pairs, keys


def work(case):
    if case["op"] == "table":
        pairs = case["count"] * case["dim"] // 2
        return {"bytes": 8 * pairs + (8 * case["count"] if case["given"] else 0), "flops": 10 * pairs}
    if case["op"] == "rows":
        rows = case["tokens"] * case["heads"]
        wide = case["dim"] if case["inplace"] else case["width"]
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": 2 * size * rows * wide + case["tokens"] * (4 * case["dim"] + 8), "flops": 3 * rows * case["dim"]}
    if case["op"] == "keep":
        moved = sum(p != i for path in paths_of(case) for i, p in enumerate(path))
        return {"bytes": 2 * moved * sum(SLOT[case["store"]]) + 4 * sum(map(len, paths_of(case))) + 12 * case["batch"], "flops": 0}
    pairs, keys = _pairs(case)
    rows = case["batch"] * case["q_len"] * case["heads"]
    return {"bytes": keys * sum(SLOT[case["store"]]) + rows * (2 * 1024 + 4), "flops": 4 * HEAD * pairs * case["heads"]}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


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


def _live_slots(case, table, lens):
    at = torch.arange(table.shape[1] * case["block"], device="cuda")
    live = at < torch.tensor(lens, device="cuda")[:, None]
    return (table.long()[:, at // case["block"]] * case["block"] + at % case["block"])[live]


def _filled(case, gen, table, total, lens, toward):
    """The cache: normalised rows of which some lean toward `toward`; slots past a request's length hold 0xff."""
    block = case["block"]
    data_bytes, scale_bytes = SLOT[case["store"]]
    cache = torch.empty(total, block * (data_bytes + scale_bytes), dtype=torch.uint8, device="cuda")
    step = max(1, 65536 // block)
    for p in range(0, total, step):
        n = min(step, total - p)
        x = torch.randn(n, block, HEAD, generator=gen, device="cuda")
        x += torch.empty(n, block, 1, device="cuda").exponential_(5.0, generator=gen) * toward
        data, scales = encode(_rms(x), case["store"])
        cache[p:p + n, :block * data_bytes] = data.reshape(n, -1)
        cache[p:p + n, block * data_bytes:] = scales.reshape(n, -1)
    stale = torch.ones(total * block, dtype=torch.bool, device="cuda")
    stale[_live_slots(case, table, lens)] = False
    for part in _split(cache, case):
        part[stale.view(total, block)] = 255
    return cache.reshape(-1)


def _split(cache, case):
    """The data rows [pages, block, ...] and the scale rows of a cache's bytes."""
    block, (data, scale) = case["block"], SLOT[case["store"]]
    pages = cache.view(-1, block * (data + scale))
    return pages[:, :block * data].unflatten(1, (block, data)), pages[:, block * data:].unflatten(1, (block, scale))


def frequencies_of(case):
    """The angle per position of each pair, in 64 bits: theta^(-2i/dim), stretched for long contexts."""
    dim, theta, factor = case["dim"], 10000.0, case["factor"]
    if case["scaling"] == "ntk":
        theta *= factor ** (dim / (dim - 2)) if dim > 2 else factor
    plain = [theta ** (-2.0 * i / dim) for i in range(dim // 2)]
    if case["scaling"] == "linear":
        return [f / factor for f in plain]
    if case["scaling"] != "yarn":
        return plain

    def index(turns):  # the pair that turns so often over the 65536 positions of the first training
        return dim / 2 * math.log(65536 / (2 * math.pi * turns)) / math.log(theta)

    low, high = max(0, math.floor(index(32.0))), min(dim // 2 - 1, math.ceil(index(1.0)))
    high = max(high, low + 0.001)
    keep = [1 - min(1.0, max(0.0, (i - low) / (high - low))) for i in range(dim // 2)]
    return [f * k + f / factor * (1 - k) for f, k in zip(plain, keep)]


def magnitude_of(case):
    return 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "yarn" else 1.0


def prepare(case, seed):
    gen = _generator(seed)
    s = dict(case)
    if case["op"] == "table":
        positions = torch.randint(0, 4 * case["count"] + 1000000, (case["count"],), generator=gen, device="cuda") if case["given"] else None
        s.update(positions=positions, first=0 if case["given"] else seed % 1000, frequencies=frequencies_of(case),
                 out=torch.empty(case["count"], case["dim"], device="cuda"))
        return s
    if case["op"] == "rows":
        positions = torch.randint(0, 8192, (case["tokens"],), generator=gen, device="cuda")
        angles = torch.arange(8192, dtype=torch.float64, device="cuda")[:, None] * (
            10000.0 ** (-torch.arange(case["dim"] // 2, dtype=torch.float64, device="cuda") * 2 / case["dim"]))
        x = torch.randn(case["tokens"], case["heads"], case["width"], generator=gen, device="cuda").to(TYPES[case["type"]])
        s.update(x=x, positions=positions, cos_sin=torch.cat([angles.cos(), angles.sin()], 1).float(),
                 out=x if case["inplace"] else torch.empty_like(x))
        return s
    lens = lens_of(case)
    table, total = _pages(case, gen, lens)
    s.update(table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), blocks=total)
    if case["op"] == "keep":
        paths = paths_of(case)
        padded = [p + [-1] * (case["q_len"] - len(p)) for p in paths]
        s.update(cache=torch.randint(0, 256, (total * case["block"] * sum(SLOT[case["store"]]),), generator=gen, device="cuda", dtype=torch.uint8),
                 path=torch.tensor(padded, dtype=torch.int32, device="cuda"),
                 path_lens=torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"),
                 new_lens=torch.empty(case["batch"], dtype=torch.int32, device="cuda"))
        return s
    batch, q_len, heads = case["batch"], case["q_len"], case["heads"]
    toward = _rms(torch.randn(HEAD, generator=gen, device="cuda"))
    q = _rms(torch.randn(batch, q_len, heads, HEAD, generator=gen, device="cuda") + 0.5 * toward).to(torch.bfloat16)
    s.update(q=q, cache=_filled(case, gen, table, total, lens, toward), lse=torch.empty(batch, q_len, heads, device="cuda"),
             out=torch.empty_like(q), sink=torch.randn(heads, generator=gen, device="cuda") if case["sinks"] else None, tree=None)
    if case["op"] == "tree":
        # 64 bits of a token in a signed word
        s["tree"] = torch.tensor([[m - (1 << 64) if m >> 63 else m for m in t] for t in trees_of(case)], dtype=torch.int64, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms

def encode(v, store):
    """Rows [..., 512] as a cache holds them: (data bytes, scale bytes)."""
    if store == "bf16":
        return v.to(torch.bfloat16).view(torch.uint8), torch.empty(*v.shape[:-1], 0, dtype=torch.uint8, device=v.device)
    groups = v[..., :NOPE].unflatten(-1, (GROUPS, GROUP))
    mantissa, exponent = torch.frexp(groups.abs().amax(-1))      # amax = mantissa * 2^exponent, mantissa in [1/2, 1)
    s = torch.where(mantissa > 0.875, exponent - 8, exponent - 9).clamp(-120, 120)  # the least s with amax <= 448 * 2^s
    codes = (groups * torch.exp2(-s.float())[..., None]).flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
    tail = v[..., NOPE:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return torch.cat([codes, tail], -1), torch.nn.functional.pad((s + 127).to(torch.uint8), (0, 1))


def decode(data, scales, store):
    """The fp32 values of rows held as bytes."""
    if store == "bf16":
        return data.contiguous().view(torch.bfloat16).float()
    codes = data[..., :NOPE].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (GROUPS, GROUP))
    exponent = scales[..., :GROUPS].int()
    step = torch.where(exponent == 0, 0x00400000, exponent << 23).view(torch.float32)  # 2^(exponent - 127)
    return torch.cat([(codes * step[..., None]).flatten(-2), data[..., NOPE:].contiguous().view(torch.bfloat16).float()], -1)


def _seen(s):
    """The mask [B, Q, L] of what each token sees."""
    at = torch.arange(s["table"].shape[1] * s["block"], device="cuda")
    q_len = s["q"].shape[1]
    c = s["lens"].long()[:, None, None] - q_len
    if s["tree"] is None:
        to = c + 1 + torch.arange(q_len, device="cuda")[:, None]
        since = to - s["window"] if s["window"] else 0
        return (at < to) & (at >= since)
    bits = s["tree"][:, :, None] >> torch.arange(64, device="cuda") & 1
    depth = bits.sum(-1, keepdim=True)
    since = c + depth - s["window"] if s["window"] else 0
    context = (at < c) & (at >= since) & (depth > 0)
    drafted = bits.gather(2, (at - c).clamp(0, 63).expand(-1, q_len, -1)) > 0
    return context | (drafted & (at >= c) & (at < c + q_len))


def attention(s):
    cache_data, cache_scales = _split(s["cache"], s)
    pages = s["table"].clamp(min=0)
    rows = decode(cache_data[pages], cache_scales[pages], s["store"]).flatten(1, 2)
    at = torch.arange(rows.shape[1], device="cuda")
    rows = torch.where((at < s["lens"][:, None])[..., None], rows, 0.0)
    scores = torch.matmul(s["q"].float().flatten(1, 2), rows.transpose(1, 2)).unflatten(1, s["q"].shape[1:3])
    scores = (scores * SOFTMAX_SCALE).masked_fill(~_seen(s)[:, :, None], -math.inf)
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
    return {"out": out.to(torch.bfloat16), "lse": (most + torch.log(total)).squeeze(-1)}


def keep(s):
    c = s["lens"].long()[:, None] - s["path"].shape[1]
    live = torch.arange(s["path"].shape[1], device="cuda") < s["path_lens"][:, None]
    b, i = torch.nonzero(live, as_tuple=True)
    src, dst = (c[:, 0][b] + s["path"].long()[b, i]), c[:, 0][b] + i
    block, table = s["block"], s["table"].long()
    for part in _split(s["cache"], s):
        part[table[b, dst // block], dst % block] = part[table[b, src // block], src % block]
    new_lens = torch.where(s["lens"] > 0, c[:, 0] + s["path_lens"], 0).int()
    return {"cache": s["cache"], "lens": new_lens}


def table(s):
    # in 64 bits: the angles of far positions
    at = s["positions"] if s["given"] else torch.arange(s["first"], s["first"] + s["count"], device="cuda")
    angles = at.double()[:, None] * torch.tensor(s["frequencies"], dtype=torch.float64, device="cuda")
    return (torch.cat([angles.cos(), angles.sin()], 1) * magnitude_of(s)).float()


def rows(s):
    x, dim, offset = s["x"], s["dim"], s["offset"]
    cos, sin = s["cos_sin"][s["positions"]][:, None].chunk(2, -1)
    if s["inverse"]:
        sin = -sin
    part = x[..., offset:offset + dim].float()
    a, b = (part[..., 0::2], part[..., 1::2]) if s["layout"] == "pairs" else part.chunk(2, -1)
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if s["layout"] == "pairs" else torch.cat(turned, -1)
    if s["inplace"]:
        x[..., offset:offset + dim] = turned.to(x.dtype)
        return x
    return torch.cat([x[..., :offset], turned.to(x.dtype), x[..., offset + dim:]], -1)


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return {"attention": attention, "tree": attention, "keep": keep, "table": table, "rows": rows}[s["op"]](s)
    import kv_norm_rope_gb300 as k
    if s["op"] == "table":
        k.rope_table(s["frequencies"], s["out"], positions=s["positions"], first=s["first"], magnitude=magnitude_of(s))
        return s["out"]
    if s["op"] == "rows":
        k.rope_rows(s["x"], s["positions"], s["cos_sin"], out=s["out"], offset=s["offset"], inverse=s["inverse"],
                    layout=k.ROPE_PAIRS if s["layout"] == "pairs" else k.ROPE_HALF)
        return s["out"]
    store = {"fp8": k.STORE_FP8, "bf16": k.STORE_BF16, "fp4": k.STORE_FP4, "indexer": k.STORE_INDEXER}[s["store"]]
    if s["op"] == "keep":
        k.tree_keep(store, s["cache"], s["blocks"], s["block"], s["table"], s["lens"], s["path"], s["path_lens"], s["new_lens"])
        return {"cache": s["cache"], "lens": s["new_lens"]}
    k.latent_attention(store, s["q"], s["cache"], s["blocks"], s["block"], s["table"], s["lens"], SOFTMAX_SCALE, s["out"],
                       lse=s["lse"], sinks=s["sink"], window=s["window"], tree=s["tree"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- in 64 bits

def _exact_values(s, pages):
    """The rows of these pages in float64, codes through a table of the bytes' values."""
    block, (data_bytes, scale_bytes) = s["block"], SLOT[s["store"]]
    raw = s["cache"].view(-1, block * (data_bytes + scale_bytes))[pages.long()]
    data = raw[:, :block * data_bytes].reshape(-1, data_bytes)
    if s["store"] == "bf16":
        return data.view(torch.bfloat16).double()
    value = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = math.ldexp(m / 8, -6) if e == 0 else math.ldexp(1 + m / 8, e - 7)
        value.append(math.nan if c & 127 == 127 else -v if c & 128 else v)
    value = torch.tensor(value, dtype=torch.float64, device="cuda")[data[:, :NOPE].long()]
    scales = raw[:, block * data_bytes:].reshape(-1, scale_bytes)[:, :GROUPS]
    value *= torch.pow(2.0, scales.double() - 127).repeat_interleave(GROUP, dim=1)
    return torch.cat([value, data[:, NOPE:].contiguous().view(torch.bfloat16).double()], 1)


def _exact_attention(s):
    q_len, trees = s["q"].shape[1], None if s["tree"] is None else s["tree"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    sink = None if s["sink"] is None else s["sink"].double()[:, None]
    for b, n in enumerate(s["lens"].tolist()):
        keys = _exact_values(s, s["table"][b][:-(-n // s["block"])])[:n]
        c = n - q_len
        for j in range(q_len):
            if trees is None:
                to, chosen = max(0, c + 1 + j), []
                since = max(0, to - s["window"]) if s["window"] else 0
            else:
                chosen = [c + i for i in range(q_len) if trees[b][j] >> i & 1 and c + i >= 0]
                depth = bin(trees[b][j] & (1 << 64) - 1).count("1")
                to = max(0, c) if depth else 0
                since = min(to, max(0, c + depth - s["window"])) if s["window"] else 0
            mine = keys[since:to] if not chosen else torch.cat([keys[since:to], keys[chosen]])
            x = s["q"][b, j].double() @ mine.T * SOFTMAX_SCALE
            if sink is not None:
                x = torch.cat([x, sink], 1)
            if x.shape[1]:
                lse[b, j] = torch.logsumexp(x, 1)
                out[b, j] = torch.softmax(x, 1)[:, :mine.shape[0]] @ mine
    return {"out": out, "lse": lse}


def _exact_table(s):
    # exp(i p f) with p = 1024 h + l, as a product
    at = s["positions"] if s["given"] else torch.arange(s["first"], s["first"] + s["count"], device="cuda")
    f = torch.tensor(s["frequencies"], dtype=torch.float64, device="cuda")
    one = torch.ones((), dtype=torch.float64, device="cuda")
    turn = torch.polar(one, (at // 1024 * 1024).double()[:, None] * f) * torch.polar(one, (at % 1024).double()[:, None] * f)
    return torch.view_as_real(turn * magnitude_of(s)).permute(0, 2, 1).flatten(1)


def _exact_rows(s):
    x, dim, offset = s["x"].double(), s["dim"], s["offset"]
    turn = torch.complex(*s["cos_sin"].double()[s["positions"]].chunk(2, 1))[:, None]
    turn = turn.conj() if s["inverse"] else turn
    part = x[..., offset:offset + dim]
    if s["layout"] == "pairs":
        part = torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(part[..., :dim // 2].contiguous(), part[..., dim // 2:].contiguous()) * turn
        part = torch.cat([z.real, z.imag], -1)
    return torch.cat([x[..., :offset], part, x[..., offset + dim:]], -1)


def exact(case, seed):
    if case["op"] == "keep":
        return None  # nothing is computed: copies and lengths
    s = prepare(case, seed)
    return {"table": _exact_table, "rows": _exact_rows}.get(case["op"], _exact_attention)(s)
