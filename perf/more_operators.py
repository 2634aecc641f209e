"""Serving from a paged cache held in 4 bits: three operators, what they are measured on, and their plain forms.

One serving step takes new tokens of b sequences, packed one sequence after another (q_starts[s] is the first row
of sequence s); kv_lengths[s] counts the positions of sequence s, its new tokens included, so new token i of n sits
at position kv_lengths[s] - n + i.  The positions lie in pages that a table [b, pages_per_seq] assigns.

A row of d keys or values is held in blocks of 16 columns: a scale s in 8 bits (e4m3: nearest, ties to even, at most
448) of the block's largest |x| / 6, and each x / s in 4 bits (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign; nearest,
ties to even), in units of 2^exp.  A page [page, 9 d / 16] of bytes has the codes of its rows first (columns 2 i and
2 i + 1 in the low and the high half of a byte), and then their scales.
  append     rotates the new queries and keys by their positions, stores keys and values into the pages in 4 bits,
             and reads the stored rows back, as a prompt's attention does that is to see what later steps will see
  read       the last n positions of each sequence as bf16 rows
  attention  softmax(scale q k^T) v of each new token over its sequence's positions up to its own, with a window
             only the last `window` of them and the first `sinks`; query head x reads key-value head x // (h / h_kv)

Head shapes are the base model's (64 wide, 8 heads), the big model's (64 wide, 16 heads) and the long causal
workload's (128 wide, 16 heads), with as many or fewer key-value heads; caches go up to that workload's 8192
positions and far beyond it.
"""
import math

import torch

own = False

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _case(name, op, b, prompts, new_lo, new_hi, len_lo, len_hi, h, h_kv, d, page, d_rot=0, interleaved=False,
          packed=False, window=0, sinks=0, v_exp=-3):
    c = {"op": op, "b": b, "prompts": prompts, "new_lo": new_lo, "new_hi": new_hi, "len_lo": len_lo,
         "len_hi": len_hi, "h": h, "h_kv": h_kv, "d": d, "page": page, "d_rot": d_rot, "interleaved": interleaved,
         "packed": packed, "window": window, "sinks": sinks, "v_exp": v_exp}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token for each of 8 chats with a base model: the launches are all there is
        _case("append_step_b8", "append", 8, 0, 1, 1, 20, 500, 8, 8, 64, 16, 64),
        # odd prompts of a few hundred tokens, half of each head rotated in neighbouring pairs, rows cut out of the
        # packed result of one projection
        _case("append_ragged", "append", 7, 7, 33, 601, 0, 900, 16, 8, 64, 32, 32, True, True),
        # two prompts of 8192 tokens
        _case("append_prompt", "append", 2, 2, 8192, 8192, 0, 0, 16, 4, 128, 64, 128),
        # the last 1 to 200 positions of 9 chats, on their way to another cache
        _case("read_b9", "read", 9, 9, 1, 200, 20, 500, 8, 8, 64, 16),
        # whole caches of 32 sequences of 4096 to 8192 positions
        _case("read_b32", "read", 32, 32, 4096, 8192, 0, 0, 16, 4, 128, 64),
        # one token of one short chat: latency
        _case("step_b1_short", "attention", 1, 0, 1, 1, 300, 300, 8, 8, 64, 16),
        # one token for each of 32 sequences over 4096 to 8192 cached positions
        _case("step_b32", "attention", 32, 0, 1, 1, 4096, 8192, 16, 4, 128, 64),
        # one sequence of 131072 positions
        _case("step_long", "attention", 1, 0, 1, 1, 131072, 131072, 16, 2, 128, 64),
        # four drafted tokens to verify for each of 16 sequences, a key-value head for each query head
        _case("verify_b16", "attention", 16, 16, 4, 4, 1000, 4001, 16, 16, 64, 32),
        # chunks of 512 prompt tokens behind 7680 cached positions
        _case("chunk_b4", "attention", 4, 4, 512, 512, 8192, 8192, 16, 4, 128, 64),
        # one token for each of 64 long chats of which the last 1024 positions and the first 4 stay visible
        _case("window_step_b64", "attention", 64, 0, 1, 1, 2000, 32768, 16, 4, 128, 64, window=1024, sinks=4),
        # two odd prompts among single tokens with such a window, three query heads to a key-value head
        _case("window_mixed_b24", "attention", 24, 2, 401, 1801, 60, 5001, 24, 8, 64, 16, window=1000, sinks=20),
    ]


def _spread(i, lo, hi, step):
    return lo + int((hi - lo + 1) * ((i * step + 0.37) % 1.0))


def _sizes(c):
    """New tokens (rows to read) and lengths of each sequence: a fixed spread over the case's ranges."""
    new, lens = [], []
    for i in range(c["b"]):
        n = _spread(i, c["new_lo"], c["new_hi"], 0.618034) if i < c["prompts"] else 1
        new.append(n)
        lens.append(max(n, _spread(i, c["len_lo"], c["len_hi"], 0.754878)))
    return new, lens


def _seen_by(c, pos):
    """Positions that the token at `pos` sees."""
    n = pos + 1
    return n if not c["window"] else min(n, c["window"]) + max(0, min(c["sinks"], n - c["window"]))


def _pairs(c):
    """Visible (token, key) pairs of one head."""
    new, lens = _sizes(c)
    if not c["window"]:
        return sum(n * (s - n) + n * (n + 1) // 2 for n, s in zip(new, lens))
    return sum(_seen_by(c, p) for n, s in zip(new, lens) for p in range(s - n, s))


def _visible(c):
    """Cached positions that some token sees, over all sequences."""
    total = 0
    for n, s in zip(*_sizes(c)):
        first = max(0, s - n - c["window"] + 1) if c["window"] else 0
        total += s - first + min(c["sinks"], first)
    return total


def _padded(c):
    new, lens = _sizes(c)
    return c["b"] * c["h"] * max(new) * max(lens)


def work(case):
    c = case
    new, lens = _sizes(c)
    t, h, h_kv, d, page = sum(new), c["h"], c["h_kv"], c["d"], c["page"]
    row, held = 2 * h_kv * d * 2, 2 * h_kv * d * 9 // 16      # a position's keys and values in bf16, and as held
    entries = 4 * (t // page + 3 * c["b"])
    if c["op"] == "append":
        return {"bytes": 2 * t * h * d * 2 + t * (2 * row + held) + entries,
                "flops": t * (3 * (h + h_kv) * c["d_rot"] + 4 * h_kv * d)}
    if c["op"] == "read":
        return {"bytes": t * (row + held) + entries, "flops": 2 * t * h_kv * d}
    seen = _visible(c)
    return {"bytes": 2 * t * h * d * 2 + seen * held + 4 * (seen // page + 3 * c["b"]), "flops": 4 * d * h * _pairs(c)}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    ops = ("append", "read", "attention")
    most = max(_padded(c) for c in listed() if c["op"] == "attention")
    top = {op: [max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")] for op in ops}
    while True:
        op = rng.choice(["append", "read", "attention", "attention", "attention"])
        h_kv, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8, 16])
        d = rng.choice([16, 32, 64, 64, 128, 128, 256])
        b = _log(rng, 1, 128)
        kind = rng.choice(["step", "few", "chunk", "mixed"])
        new_hi = {"step": 1, "few": rng.randint(2, 8), "chunk": _log(rng, 9, 8192), "mixed": _log(rng, 9, 2048)}[kind]
        new_lo = rng.randint(1, new_hi)
        prompts = {"step": 0, "few": b, "chunk": b, "mixed": max(1, b // 8)}[kind]
        len_hi = _log(rng, max(1, new_hi // 2), 131072)
        c = _case(None, op, b, prompts, new_lo, new_hi, rng.randint(1, len_hi), len_hi, h_kv * group, h_kv, d,
                  rng.choice([16, 32, 64, 128, 256]), v_exp=rng.choice([-5, -3, 0]))
        if op == "append":
            c["d_rot"] = rng.choice([0, 16, d // 2 // 16 * 16, d, d])
            c["interleaved"], c["packed"] = rng.random() < 0.5, rng.random() < 0.5
        if op == "attention" and rng.random() < 0.5:
            c["window"], c["sinks"] = _log(rng, 1, 8192), rng.choice([0, 1, 4, 16, 100])
        if op != "attention":
            c["len_lo"], c["len_hi"] = min(c["len_lo"], 2000), min(c["len_hi"], 2000)
        w = work(c)
        cached = sum(_sizes(c)[1]) * h_kv * d
        if (c["h"] <= 64 and cached <= 1 << 28 and w["bytes"] <= top[op][0] and w["flops"] <= top[op][1]
                and (op != "attention" or _padded(c) <= most)):
            return c


def _scale_codes(x, exp):
    """The scales (e4m3, as their values) and codes (0 .. 15) of x [..., d] in fp64, in units of 2^exp."""
    x = (x * 2.0 ** -exp).unflatten(-1, (-1, 16))
    s = (x.abs().amax(-1) / 6).clamp(max=448.0)
    step = torch.exp2(torch.frexp(s).exponent.clamp(min=-5).to(x.dtype) - 4)   # e4m3's at s: 3 bits of fraction
    s = (torch.round(s / step) * step).to(torch.float8_e4m3fn)
    v = s.to(x.dtype)[..., None]
    y = torch.where(v > 0, x.abs() / v, 0.0)
    # ties go to the even code
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = code.to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)
    return s, code.flatten(-2)


def _held(x, exp):
    """The bytes that rows x [..., d] are held in: codes [..., d / 2] and scales [..., d / 16]."""
    s, code = _scale_codes(x, exp)
    return code[..., 0::2] | code[..., 1::2] << 4, s.view(torch.uint8)


def _parts(pages, d):
    """Views of the codes [n, h_kv, page, d / 2] and scales [n, h_kv, page, d / 16] of pages."""
    page = pages.shape[2]
    flat, n = pages.flatten(2), page * d // 2
    return flat[..., :n].unflatten(-1, (page, d // 2)), flat[..., n:].unflatten(-1, (page, d // 16))


def _values(codes, scales, exp, dtype=torch.float32):
    grid = torch.tensor(GRID + [-x for x in GRID], dtype=dtype, device=codes.device)
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    x = grid[x.int()].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).to(dtype)[..., None]
    return (x * 2.0 ** exp).flatten(-2)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    new, lens = _sizes(c)
    b, t, h, h_kv, d, page = c["b"], sum(new), c["h"], c["h_kv"], c["d"], c["page"]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # keys have channels that are larger than others, values are small
    gains = torch.exp(0.5 * normal(h_kv, d))

    def keys(n):
        return (normal(n, h_kv, d) * gains).bfloat16()

    def values(n):
        return (0.2 * normal(n, h_kv, d)).bfloat16()

    # pages are handed out in no order; entries past a sequence's last page are never read, nor are those of pages
    # that have left the window, which are given back
    need = [-(-s // page) for s in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((b, max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
        if c["window"]:
            first = max(0, lens[s] - new[s] - c["window"] + 1)
            table[s, -(-min(c["sinks"], first) // page):first // page] = -1
    starts = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    s = {"case": c, "max_new": max(new), "table": table.to(dev), "starts": starts.to(dev),
         "lengths": torch.tensor(lens, dtype=torch.int32, device=dev)}
    for name, make, exp in (("k_pages", keys, 0), ("v_pages", values, c["v_exp"])):
        codes, scales = _held(make(n_pages * page).float(), exp)
        s[name] = torch.cat([x.unflatten(0, (n_pages, page)).transpose(1, 2).flatten(2) for x in (codes, scales)],
                            -1).unflatten(-1, (page, 9 * d // 16)).contiguous()
    if c["op"] == "append":
        q, k, v = normal(t, h, d).bfloat16(), keys(t), values(t)
        if c["packed"]:   # [t, (h + 2 h_kv) d], the rows of one projection
            rows = torch.cat((q, k, v), 1)
            q, k, v = rows[:, :h], rows[:, h:h + h_kv], rows[:, h + h_kv:]
        s["q"], s["k"], s["v"] = q, k, v
        if c["d_rot"]:
            i = torch.arange(0, c["d_rot"], 2, dtype=torch.float64)
            s["freqs"] = (10000.0 ** (-i / c["d_rot"])).float().to(dev)
        else:
            s["freqs"] = None
        s["q_out"] = torch.empty(t, h, d, dtype=torch.bfloat16, device=dev)
    elif c["op"] == "attention":
        s["q"] = normal(t, h, d).bfloat16()
        s["out"] = torch.empty(t, h, d, dtype=torch.bfloat16, device=dev)
    if c["op"] != "attention":
        s["k_out"] = torch.empty(t, h_kv, d, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty(t, h_kv, d, dtype=torch.bfloat16, device=dev)
    return s


def _tokens(s, t):
    """Sequence and position of every packed row."""
    starts = s["starts"].long()
    i = torch.arange(t, device=starts.device)
    seq = torch.searchsorted(starts, i, right=True) - 1
    return seq, s["lengths"].long()[seq] - starts[seq + 1] + i


def _rotate(x, cos, sin, interleaved):
    x = x.double()
    n = 2 * cos.shape[-1]
    if not n:
        return x
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if interleaved else (x[..., :n // 2], x[..., n // 2:n])
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    return torch.cat((r, x[..., n:]), -1)


def _plain_read(s):
    c = s["case"]
    seq, pos = _tokens(s, s["k_out"].shape[0])
    at = s["table"][seq, pos // c["page"]].long()
    for name, exp in (("k", 0), ("v", c["v_exp"])):
        codes, scales = (x[at, :, pos % c["page"]] for x in _parts(s[name + "_pages"], c["d"]))
        s[name + "_out"].copy_(_values(codes, scales, exp))
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_append(s):
    c = s["case"]
    seq, pos = _tokens(s, s["q"].shape[0])
    n = c["d_rot"] // 2
    # 64 bits: angles of far positions, and values next to the border of two codes
    angle = pos.double()[:, None, None] * (s["freqs"].double() if n else pos.new_zeros(0).double())
    cos, sin = angle.cos(), angle.sin()
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["interleaved"]))
    at = s["table"][seq, pos // c["page"]].long()
    for name, x, exp in (("k_pages", _rotate(s["k"], cos, sin, c["interleaved"]), 0),
                         ("v_pages", s["v"].double(), c["v_exp"])):
        for part, held in zip(_parts(s[name], c["d"]), _held(x, exp)):
            part[at, :, pos % c["page"]] = held
    return dict(_plain_read(s), q=s["q_out"])


def _plain_attention(s):
    c = s["case"]
    b, h_kv, d, n = c["b"], c["h_kv"], c["d"], s["max_new"]
    g = c["h"] // h_kv
    starts, lens = s["starts"].long(), s["lengths"].long()
    new = starts[1:] - starts[:-1]
    at = s["table"].long().clamp(min=0)

    def cached(pages, exp):   # [b, h_kv, positions, d]
        return _values(*(x[at].transpose(1, 2).flatten(2, 3) for x in _parts(pages, d)), exp)

    i = torch.arange(n, device=at.device)
    q = s["q"][(starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()         # [b, n, h, d]
    q = q.view(b, n, h_kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, h_kv, g * n, d)
    x = torch.matmul(q, cached(s["k_pages"], 0).transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    j = torch.arange(x.shape[-1], device=at.device)
    pos = ((lens - new)[:, None] + i)[..., None]
    seen = j <= pos                                                                     # [b, n, positions]
    if c["window"]:
        seen &= (j > pos - c["window"]) | (j < c["sinks"])
    x = x.view(b, h_kv, g, n, -1).masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)))
    p = p.masked_fill_(~seen[:, None, None], 0.0)
    o = torch.matmul(p.view(b, h_kv, g * n, -1), cached(s["v_pages"], c["v_exp"]))
    o = o / p.sum(-1).clamp(min=1e-30).view(b, h_kv, g * n, 1)
    o = o.view(b, h_kv * g, n, d)
    seq, pos = _tokens(s, s["q"].shape[0])
    s["out"].copy_(o[seq, :, pos - (lens - new)[seq]])
    return {"out": s["out"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention}[c["op"]](s)
    import transformer_scaled_dot_02_gb300 as sd
    if c["op"] == "attention":
        if "workspace" not in s:   # a serving loop keeps one
            s["workspace"] = sd.paged4_workspace(s["q"], s["k_pages"], s["table"])
        sd.paged4_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["starts"], s["lengths"],
                            v_exp=c["v_exp"], window=c["window"], sinks=c["sinks"], out=s["out"],
                            workspace=s["workspace"])
        return {"out": s["out"]}
    if c["op"] == "append":
        sd.paged4_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["starts"], s["lengths"],
                         rope_freqs=s["freqs"], interleaved=c["interleaved"], v_exp=c["v_exp"], q_out=s["q_out"])
    sd.paged4_read(s["k_pages"], s["v_pages"], s["table"], s["starts"], s["lengths"], s["k_out"], s["v_out"],
                   v_exp=c["v_exp"])
    return dict({"k": s["k_out"], "v": s["v_out"]}, **({"q": s["q_out"]} if c["op"] == "append" else {}))


def _nearest(x, grid):
    """The element of the increasing `grid` nearest to x >= 0; of two as near, the one of even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    return grid[torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)]


def _as_held(x, exp):
    """What rows in fp64 stand for once they are held in 4 bits."""
    # every finite e4m3 number from zero on: 3 bits of fraction, exponents from 2^-6 on
    e4m3 = [m / 8 * 2.0 ** -6 for m in range(8)]
    e4m3 += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)]
    x = x.unflatten(-1, (-1, 16)) / 2.0 ** exp
    s = _nearest(x.abs().amax(-1, keepdim=True) / 6, e4m3)
    y = _nearest(torch.nan_to_num(x.abs() / s, nan=0.0, posinf=0.0), GRID)
    return (torch.sign(x) * y * s * 2.0 ** exp).flatten(-2)


def _stored(pages, d, at, head, rows, exp):
    """Positions 0 .. rows - 1 of a sequence with pages `at`, one key-value head, in fp64."""
    page = pages.shape[2]
    x = pages[at, head].reshape(len(at), -1).int()
    codes = x[:, :page * d // 2].reshape(-1, d // 2)[:rows]
    scales = x[:, page * d // 2:].reshape(-1, d // 16)[:rows]
    e, m = scales >> 3, (scales & 7).double()
    s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
    out = torch.empty(rows, d, dtype=torch.float64, device=pages.device)
    for half in range(2):
        c = codes >> 4 * half & 15
        mag, low = c >> 1 & 3, (c & 1).double()
        v = torch.where(mag > 0, (1 + low / 2) * torch.exp2(mag.double() - 1), low / 2)
        out[:, half::2] = torch.where(c >= 8, -v, v)
    return out * s.repeat_interleave(16, 1) * 2.0 ** exp


def exact(case, seed):
    """The definitions, sequence by sequence and in 64 bits."""
    s = prepare(case, seed)
    c = case
    new, lens = _sizes(c)
    h, h_kv, d, page = c["h"], c["h_kv"], c["d"], c["page"]
    dev = s["table"].device
    table = s["table"].cpu().tolist()
    if c["op"] == "append":
        x = {name: s[name].double() for name in ("q", "k", "v")}
        t = 0
        for n, length in zip(new, lens):
            if c["d_rot"]:
                pos = torch.arange(length - n, length, device=dev)
                turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev),
                                   pos.double()[:, None] * s["freqs"].double())[:, None]
                for name in ("q", "k"):
                    part = x[name][t:t + n, :, :c["d_rot"]]
                    m = c["d_rot"] // 2
                    a, b = (slice(0, None, 2), slice(1, None, 2)) if c["interleaved"] else (slice(m), slice(m, None))
                    z = torch.complex(part[..., a], part[..., b]) * turn
                    part[..., a], part[..., b] = z.real, z.imag
            t += n
        return {"q": x["q"], "k": _as_held(x["k"], 0), "v": _as_held(x["v"], c["v_exp"])}
    t = 0
    if c["op"] == "read":
        out = {x: torch.empty(sum(new), h_kv, d, dtype=torch.float64, device=dev) for x in ("k", "v")}
        for n, length, pages in zip(new, lens, table):
            at = torch.tensor(pages[:-(-length // page)], device=dev)
            for x in range(h_kv):
                out["k"][t:t + n, x] = _stored(s["k_pages"], d, at, x, length, 0)[length - n:]
                out["v"][t:t + n, x] = _stored(s["v_pages"], d, at, x, length, c["v_exp"])[length - n:]
            t += n
        return out
    out = torch.empty(sum(new), h, d, dtype=torch.float64, device=dev)
    for n, length, pages in zip(new, lens, table):
        at = torch.tensor(pages[:-(-length // page)], device=dev).clamp(min=0)
        pos, j = torch.arange(length - n, length, device=dev)[:, None], torch.arange(length, device=dev)[None]
        hidden = j > pos
        if c["window"]:
            hidden |= (j <= pos - c["window"]) & (j >= c["sinks"])
        for y in range(h_kv):
            k = _stored(s["k_pages"], d, at, y, length, 0)
            v = _stored(s["v_pages"], d, at, y, length, c["v_exp"])
            for x in range(y * (h // h_kv), (y + 1) * (h // h_kv)):
                w = s["q"][t:t + n, x].double() @ k.T / math.sqrt(d)
                out[t:t + n, x] = torch.softmax(w.masked_fill(hidden, -math.inf), -1) @ v
        t += n
    return {"out": out}
