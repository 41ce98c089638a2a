"""The operators that make and shape the rows a verifier reads, as cases to measure.

A verification round runs the target model over N = gamma + 1 rows of every
request; row j of request b stands at position kv_len[b] + j. Around the verifier
itself that needs

  rotate  spec_verify_rotate: rotary positions of queries and keys. With
          a_i = (kv_len + j) f_i the pair (x, y) of dimensions (i, i + R/2) or
          (2i, 2i + 1) becomes m (x cos a - y sin a), m (y cos a + x sin a).
  write   spec_verify_cache_write: the rows' keys and values into a paged cache of
          e4m3 codes, with one scale for each block of 32 tokens and head: the
          smallest power of two 2^e with max |x| <= 448 2^e over the block's content.
          Rows that the block held before are taken over at the new scale.
  read    spec_verify_cache_read: code times scale, of a range of positions.
  attend  spec_verify_attention: softmax(s q k) v over the cache's codes times scales,
          a row seeing positions max(0, p - window + 1) .. p, p its own.
  adjust  spec_verify_adjust_logits: repetition, frequency and presence penalties of
          the tokens before a row, biases, and a grammar's mask.

A block of 32 tokens of one head is stored as bricks of 32 dimensions, 1,024 bytes each,
in the order in which a wave's lanes take a matrix instruction's operand:
  keys    byte 256 (d / 8) + 16 (4 (s / 8) + s % 4) + 8 (s / 4 % 2) + d % 8,
  values  byte 256 (s / 8) + 16 (d % 16) + 8 (d / 16) + s % 8,
for token s of the block and dimension d of the brick.

`run` is one pass, in plain torch operations where `own` is false and through
the package's entry points where it is true.
"""

import random

import torch

own = False

BLOCK = 32


def listed():
    """Batches, draft lengths and vocabularies are those of the benchmark's configurations."""
    return [
        # a verification round's queries and keys: 128 requests of nine rows, 32 and 8 heads of 128
        dict(name="rotate_round", op="rotate", B=128, N=9, Hq=32, Hk=8, D=128, R=128, inter=False,
             dtype="bf16", L=8192, fused=False, stretch=1.0),
        # prompts in float32 at far positions, half of each head rotated in neighbouring pairs, cut from one
        # fused projection
        dict(name="rotate_prompt_f32", op="rotate", B=3, N=1531, Hq=12, Hk=4, D=96, R=48, inter=True,
             dtype="f32", L=120000, fused=True, stretch=4.0),
        # the same round's keys and values, and the blocks they changed
        dict(name="write_round", op="write", B=128, N=9, H=8, D=128, page=64, dtype="bf16", L=4096, rows=False),
        # prompts of up to 4,096 tokens: requests of different lengths in one padded batch
        dict(name="write_prompt", op="write", B=4, N=4096, H=8, D=128, page=128, dtype="bf16", L=0, rows=True),
        # a long prefix read back, to be handed to another worker
        dict(name="read_prefix", op="read", B=2, L=32768, H=8, D=128, page=64, dtype="bf16"),
        # a few short requests in float32, heads of 80
        dict(name="read_few_f32", op="read", B=3, L=701, H=5, D=80, page=32, dtype="f32"),
        # one new token of one request
        dict(name="attend_one_token", op="attend", B=1, N=1, Hq=32, H=8, D=128, page=64, low=1000, L=1000,
             dtype="bf16", window=0, rows=False),
        # a round of a ragged batch: nine rows a request over 100 to 8,192 tokens
        dict(name="attend_round", op="attend", B=128, N=9, Hq=32, H=8, D=128, page=64, low=100, L=8192,
             dtype="bf16", window=0, rows=False),
        # few requests with long contexts: five rows, groups of eight query heads
        dict(name="attend_long", op="attend", B=4, N=5, Hq=64, H=8, D=128, page=128, low=131072, L=131072,
             dtype="bf16", window=0, rows=False),
        # float32, heads of 80 that share nothing, a sliding window, requests of fewer rows
        dict(name="attend_f32_window", op="attend", B=7, N=6, Hq=6, H=6, D=80, page=32, low=1, L=5003,
             dtype="f32", window=1000, rows=True),
        # every row of a verified batch under a grammar, with penalties and biases
        dict(name="adjust_round", op="adjust", B=128, N=9, V=151936, dtype="bf16", pad=0, history=600, prompt=1400,
             bias=64, mask=True),
        # one request's rows in float32, an odd vocabulary, cut from a padded buffer; penalties and biases only
        dict(name="adjust_request_f32", op="adjust", B=1, N=5, V=50257, dtype="f32", pad=47, history=333,
             prompt=0, bias=7, mask=False),
    ]


def _log_int(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["rotate", "write", "read", "attend", "attend", "attend", "adjust", "adjust"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([32, 64, 128, 256])
    D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256, rng.randint(8, 256)])
    if op == "rotate":
        Hk, B = rng.randint(1, 8), _log_int(rng, 1, 256)
        Hq, D = Hk * rng.randint(1, 8), D // 2 * 2
        N = _log_int(rng, 1, max(1, min(4096, 150_000_000 // (B * (Hq + Hk) * D))))
        return dict(op=op, B=B, N=N, Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D, 2 * rng.randint(1, D // 2)]),
                    inter=rng.random() < 0.5, dtype=dtype, L=_log_int(rng, 1, 131072), fused=rng.random() < 0.5,
                    stretch=round(rng.uniform(1.0, 8.0), 2))
    H = rng.randint(1, 8)
    if op == "write":
        B = _log_int(rng, 1, 128)
        N = _log_int(rng, 1, max(1, min(8192, 16_000_000 // (B * H * D))))
        return dict(op=op, B=B, N=N, H=H, D=D, page=page, dtype=dtype, L=_log_int(rng, 1, 1 + 4096 // B),
                    rows=rng.random() < 0.5)
    if op == "read":
        B = _log_int(rng, 1, 64)
        return dict(op=op, B=B, L=_log_int(rng, 1, max(1, min(65536, 67_000_000 // (B * H * D)))), H=H, D=D, page=page,
                    dtype=dtype)
    if op == "attend":
        B, N = _log_int(rng, 1, 128), rng.choice([1, rng.randint(2, 9), _log_int(rng, 1, 64)])
        Hq = H * rng.randint(1, 8)
        # the cache and the products within the largest listed ones
        L = _log_int(rng, 1, max(1, min(131072, 500_000_000 // (B * H * D), 19_000_000_000 // (B * N * Hq * D))))
        return dict(op=op, B=B, N=N, Hq=Hq, H=H, D=D, page=page, low=rng.choice([L, max(1, L // 8), 1]), L=L,
                    dtype=dtype, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), rows=rng.random() < 0.4)
    V = min(151936, rng.choice([_log_int(rng, 1000, 151936), 32000, 50257, 128256, 151936]))
    B = _log_int(rng, 1, 256)
    N = min(rng.randint(1, 16), max(1, 1152 // B // (1 if dtype == "bf16" else 2)))
    return dict(op=op, B=B, N=N, V=V, dtype=dtype, pad=rng.choice([0, 0, 8, rng.randint(1, 99)]),
                history=rng.choice([0, _log_int(rng, 1, 8192)]), prompt=rng.choice([0, _log_int(rng, 1, 8192)]),
                bias=rng.choice([0, _log_int(rng, 1, 300)]), mask=rng.random() < 0.6)


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case, low, high):
    """Tokens of each request before the call: the same for every seed, so that a case is one amount of work."""
    rng = random.Random(1000 * case["B"] + high)
    return [rng.randint(low, high) for _ in range(case["B"])]


def _row_counts(case):
    rng = random.Random(77 * case["B"] + case["N"])
    return [rng.randint(max(1, case["N"] // 2), case["N"]) if case.get("rows") else case["N"] for _ in range(case["B"])]


def _before(case):
    """Tokens that each request holds before its rows."""
    if case["op"] == "write":
        return _lengths(case, 0, case["L"])
    if case["op"] == "read":
        return _lengths(case, case["L"] * 3 // 4, case["L"])
    return _lengths(case, case["low"], case["L"])


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _type(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def whole(low, high, *shape):
        return torch.randint(low, high, shape, generator=gen, device=dev)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    B, N = case["B"], case.get("N", 1)
    s = dict(case=case)
    if case["op"] == "rotate":
        Hq, Hk, D, R = case["Hq"], case["Hk"], case["D"], case["R"]
        s["kv_len"] = whole(0, case["L"] + 1, B).to(torch.int32)
        # a base that is raised for longer contexts, and the attention's temperature that goes with it
        base = 10000.0 * case["stretch"] ** (R / max(2, R - 2))
        s["freqs"] = base ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device=dev) / R)
        s["scale"] = 1.0 + 0.1 * (case["stretch"] - 1.0)
        if case["fused"]:
            both = normal(B, N, (Hq + 2 * Hk) * D).to(dt)
            s["q"] = both[..., : Hq * D].view(B, N, Hq, D)
            s["k"] = both[..., Hq * D: (Hq + Hk) * D].view(B, N, Hk, D)
        else:
            s["q"], s["k"] = normal(B, N, Hq, D).to(dt), normal(B, N, Hk, D).to(dt)
        return s
    if case["op"] == "adjust":
        V = case["V"]
        s["logits"] = normal(B, N, V + case["pad"]).mul_(3.0).to(dt)[..., :V]
        s["tokens"] = whole(0, V, B, N).to(torch.int32)[:, : max(N - 1, 1)].contiguous() if N > 1 else None
        # text repeats itself: ids crowd towards the vocabulary's front; padding on the left
        for name in ("history", "prompt"):
            n = case[name]
            ids = (torch.rand(B, n, generator=gen, device=dev) ** 3 * V).to(torch.int32).clamp_(max=V - 1)
            ids.masked_fill_(torch.arange(n, device=dev) < whole(0, n // 2 + 1, B, 1), -1)
            s[name] = ids if n else None
        s["repetition"] = 1.0 + torch.rand(B, generator=gen, device=dev) * 0.5
        s["frequency"] = torch.rand(B, generator=gen, device=dev) * 0.5
        s["presence"] = torch.rand(B, generator=gen, device=dev)
        n = min(case["bias"], V)
        s["bias_ids"] = torch.rand(B, V, generator=gen, device=dev).topk(n).indices.to(torch.int32) if n else None
        s["bias"] = normal(B, n).mul_(2.0) if n else None
        if case["mask"]:
            # a grammar's states: most tokens allowed, a few allowed, or no constraint at this row
            bits = [whole(-2 ** 31, 2 ** 31, B, N, -(-V // 32)) for _ in range(4)]
            kind = whole(0, 3, B, N, 1)
            most, few = bits[0] | bits[1] | bits[2] | bits[3], bits[0] & bits[1] & bits[2] & bits[3]
            s["allowed"] = torch.where(kind == 0, most, torch.where(kind == 1, few, -1)).to(torch.int32)
        else:
            s["allowed"] = None
        return s
    H, D, page = case["H"], case["D"], case["page"]
    before, counts = _before(case), _row_counts(case) if "N" in case else [0] * B
    after = [a + n for a, n in zip(before, counts)]
    width = max(1, max(-(-a // page) for a in after))
    pages, per, bricks = B * width + 3, page // BLOCK, -(-D // 32)
    table = torch.randperm(pages, generator=gen, device=dev)[: B * width].view(B, width)
    dims = torch.arange(bricks * 32, device=dev)
    k_pad = (dims >= D).view(1, 1, 1, bricks, 4, 1, 1, 8)                          # keys: [brick, d/8, ., ., d%8]
    v_pad = (dims >= D).view(1, 1, 1, bricks, 1, 2, 16, 1).transpose(5, 6)         # values: [brick, ., d%16, d/16, .]
    for name, pad, shape in (("k", k_pad, (4, 16, 2, 8)), ("v", v_pad, (4, 16, 2, 8))):
        x = normal(pages, H, per, bricks, *shape).masked_fill_(pad, 0.0)
        # heads and blocks of different sizes
        amax = x.abs().amax((3, 4, 5, 6, 7)) * torch.exp2(whole(-3, 3, pages, H, per).float())
        x = x * (448.0 / x.abs().amax((3, 4, 5, 6, 7), keepdim=True))
        scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
        s[name + "_codes"] = x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(pages, H, per, bricks, 1024)
        s[name + "_scale"] = scale
    s.update(page_table=table.to(torch.int32).contiguous(), kv_len=ints(before), before=before, counts=counts,
             rows=ints(counts) if case.get("rows") else None)
    if case["op"] == "read":
        # from the first position on; the longest request fills its rows
        s["first"], s["most"] = ints([0] * B), max(before)
        s["rows"] = ints(before)
        s["out"] = tuple(torch.zeros(B, s["most"], H, D, dtype=dt, device=dev) for _ in range(2))
    if case["op"] == "write":
        s["k"], s["v"] = normal(B, N, H, D).to(dt), normal(B, N, H, D).mul_(0.5).to(dt)
        # the blocks that the rows fall into are read back from their start
        first = [a // BLOCK * BLOCK for a in before]
        held = [a - f for a, f in zip(after, first)]
        s["first"], s["held"], s["most"] = ints(first), ints(held), max(held)
        s["out"] = tuple(torch.zeros(B, s["most"], H, D, dtype=dt, device=dev) for _ in range(2))
        s["blocks"] = torch.tensor([(b, i) for b in range(B) for i in range(first[b] // BLOCK, -(-after[b] // BLOCK))],
                                   device=dev)
    if case["op"] == "attend":
        s["q"] = normal(B, N, case["Hq"], D).to(dt)
        s["out"] = torch.zeros_like(s["q"])
    return s


def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["op"]](case, state)


# ---------------------------------------------------------------- the package


def _cache(sv, s):
    return sv.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["case"]["page"], s["case"]["D"])


def _own_rotate(case, s):
    import lossless_draft_verification_sample_amd as sv
    r = sv.spec_verify_rotate(s["q"], s["k"], s["kv_len"], s["freqs"], interleaved=case["inter"], scale=s["scale"])
    return dict(q=r.q, k=r.k)


def _own_write(case, s):
    import lossless_draft_verification_sample_amd as sv
    cache = _cache(sv, s)
    sv.spec_verify_cache_write(cache, s["page_table"], s["kv_len"], s["k"], s["v"], rows=s["rows"])
    r = sv.spec_verify_cache_read(cache, s["page_table"], s["first"], s["most"], rows=s["held"],
                                  out=sv.CacheRows(*s["out"]))
    return dict(k=r.k, v=r.v, k_scale=s["k_scale"], v_scale=s["v_scale"])


def _own_read(case, s):
    import lossless_draft_verification_sample_amd as sv
    r = sv.spec_verify_cache_read(_cache(sv, s), s["page_table"], s["first"], s["most"], rows=s["rows"],
                                  out=sv.CacheRows(*s["out"]))
    return dict(k=r.k, v=r.v)


def _own_attend(case, s):
    import lossless_draft_verification_sample_amd as sv
    out = None if s["rows"] is None else sv.AttentionOut(s["out"], None)
    r = sv.spec_verify_attention(s["q"], _cache(sv, s), s["page_table"], s["kv_len"], window=case["window"],
                                 rows=s["rows"], out=out)
    return dict(out=r.out)


def _own_adjust(case, s):
    import lossless_draft_verification_sample_amd as sv
    return dict(logits=sv.spec_verify_adjust_logits(
        s["logits"], tokens=s["tokens"], history=s["history"], prompt=s["prompt"], repetition=s["repetition"],
        frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"], allowed=s["allowed"]))


_own = dict(rotate=_own_rotate, write=_own_write, read=_own_read, attend=_own_attend, adjust=_own_adjust)


# ---------------------------------------------------------------- plain forms


def _plain_rotate(case, s):
    R, dev = case["R"], s["q"].device
    at = s["kv_len"].double()[:, None] + torch.arange(case["N"], device=dev)
    angle = at[..., None] * s["freqs"]
    cos, sin = ((f(angle) * s["scale"]).float()[:, :, None] for f in (torch.cos, torch.sin))

    def turn(x):
        y = x.float()
        lo, hi = (y[..., 0:R:2], y[..., 1:R:2]) if case["inter"] else (y[..., : R // 2], y[..., R // 2: R])
        a, b = lo * cos - hi * sin, hi * cos + lo * sin
        both = torch.stack((a, b), -1).flatten(-2) if case["inter"] else torch.cat((a, b), -1)
        return torch.cat((both, y[..., R:]), -1).to(x.dtype)

    return dict(q=turn(s["q"]), k=turn(s["k"]))


def _natural(codes, keys):
    """[..., bricks, 1024] codes as [..., 32 tokens, dimensions]."""
    lead, bricks = codes.shape[:-2], codes.shape[-2]
    n = len(lead)
    if keys:   # brick, d/8, s/8, s%4, s/4%2, d%8
        x, order = codes.reshape(*lead, bricks, 4, 4, 4, 2, 8), (2, 4, 3, 0, 1, 5)
    else:      # brick, s/8, d%16, d/16, s%8
        x, order = codes.reshape(*lead, bricks, 4, 16, 2, 8), (1, 4, 0, 3, 2)
    return x.permute(*range(n), *(n + i for i in order)).reshape(*lead, BLOCK, bricks * 32)


def _bricks(x, keys):
    """The way back."""
    lead, bricks = x.shape[:-2], x.shape[-1] // 32
    n = len(lead)
    if keys:   # s/8, s/4%2, s%4, brick, d/8, d%8
        y, order = x.reshape(*lead, 4, 2, 4, bricks, 4, 8), (3, 4, 0, 2, 1, 5)
    else:      # s/8, s%8, brick, d/16, d%16
        y, order = x.reshape(*lead, 4, 8, bricks, 2, 16), (2, 0, 4, 3, 1)
    return y.permute(*range(n), *(n + i for i in order)).reshape(*lead, bricks, 1024)


def _values(codes, scale, table, keys, D):
    """The tokens of a table's pages, [..., heads, tokens, D] for a table [..., pages]."""
    lead, (_, H, per, bricks, _) = table.shape[:-1], codes.shape
    c = codes.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn).float()    # [..., pages, heads, per, bricks, 1024]
    x = _natural(c * scale[table.long()][..., None, None], keys)
    n = len(lead)
    return x.transpose(n, n + 1).reshape(*lead, H, -1, bricks * 32)[..., :D]


def _put(codes, scale, x, keys, s, case):
    """Rows x [B, N, heads, D] into the blocks that they fall into."""
    per, D, bricks = case["page"] // BLOCK, case["D"], codes.shape[-2]
    b, i = s["blocks"].unbind(1)
    at = (i * BLOCK)[:, None] + torch.arange(BLOCK, device=x.device)                # [blocks, 32] positions
    row = at - s["kv_len"].long()[b][:, None]
    count = s["rows"].long()[b] if s["rows"] is not None else torch.full_like(b, case["N"])
    new, old = (row >= 0) & (row < count[:, None]), row < 0
    page = s["page_table"].long()[b, i // per]
    had = codes.view(torch.uint8)[page, :, i % per]                                 # [blocks, heads, bricks, 1024]
    held = had.view(torch.float8_e4m3fn).float() * scale[page, :, i % per][..., None, None]
    fresh = x[b[:, None], row.clamp(0, case["N"] - 1)].float().transpose(1, 2)      # [blocks, heads, 32, D]
    fresh = torch.nn.functional.pad(fresh, (0, bricks * 32 - D))
    y = torch.where(new[:, None, :, None], fresh, torch.where(old[:, None, :, None], _natural(held, keys), 0.0))
    fine = torch.isfinite(y)
    amax = torch.where(fine, y.abs(), 0.0).amax((2, 3))
    part, power = torch.frexp(amax)
    power = (power - 9 + (part > 0.875).int()).clamp(min=-126)
    size = torch.where(amax > 0, ((power + 127) << 23).view(torch.float32), 1.0)
    code = torch.where(fine, y / size[..., None, None], float("nan")).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = (new | old)[:, None, :, None].expand(code.shape)
    code = torch.where(_bricks(keep, keys), _bricks(code, keys), had)
    codes.view(torch.uint8)[page, :, i % per] = code
    scale[page, :, i % per] = size


def _take(s, case, first, count):
    """Positions first .. first + count - 1 of every request into the state's outputs."""
    most = s["most"]
    at = first.long()[:, None] + torch.arange(most, device=first.device)            # [B, most]
    used = (torch.arange(most, device=first.device) < count.long()[:, None])[:, :, None, None]
    per = case["page"]
    page = s["page_table"].long().gather(1, (at // per).clamp(max=s["page_table"].shape[1] - 1))
    d, t = torch.arange(case["D"], device=first.device), (at % BLOCK)[..., None]
    place = dict(k=256 * (d % 32 // 8) + 16 * (4 * (t // 8) + t % 4) + 8 * (t // 4 % 2) + d % 8,
                 v=256 * (t // 8) + 16 * (d % 16) + 8 * (d % 32 // 16) + t % 8)
    heads, block = torch.arange(case["H"], device=first.device), at % per // BLOCK
    for out, name in zip(s["out"], ("k", "v")):
        codes = s[name + "_codes"].view(torch.uint8)
        got = codes[page[:, :, None, None], heads[:, None], block[:, :, None, None], d // 32, place[name][:, :, None]]
        scale = s[name + "_scale"][page[:, :, None], heads, block[:, :, None]][..., None]
        value = got.view(torch.float8_e4m3fn).float() * scale
        out.copy_(torch.where(used, value.to(out.dtype), out))
    return s["out"]


def _plain_write(case, s):
    _put(s["k_codes"], s["k_scale"], s["k"], True, s, case)
    _put(s["v_codes"], s["v_scale"], s["v"], False, s, case)
    k, v = _take(s, case, s["first"], s["held"])
    return dict(k=k, v=v, k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_read(case, s):
    k, v = _take(s, case, s["first"], s["rows"])
    return dict(k=k, v=v)


def _plain_attend(case, s):
    B, N, H, D = case["B"], case["N"], case["H"], case["D"]
    G, dev = case["Hq"] // H, s["q"].device
    k = _values(s["k_codes"], s["k_scale"], s["page_table"], True, D)               # [B, heads, tokens, D]
    q = s["q"].float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    z = (torch.matmul(q, k.transpose(2, 3)) * D ** -0.5).view(B, H, N, G, -1)
    del k
    at = torch.arange(z.shape[-1], device=dev)
    own_at = s["kv_len"].long()[:, None] + torch.arange(N, device=dev)              # [B, N]
    seen = at <= own_at[..., None]
    if case["window"]:
        seen &= at > own_at[..., None] - case["window"]
    z.masked_fill_(~seen[:, None, :, None], float("-inf"))
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    v = _values(s["v_codes"], s["v_scale"], s["page_table"], False, D)
    o = torch.matmul(p.view(B, H, N * G, -1), v).view(B, H, N, G, D)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D).to(s["q"].dtype)
    if s["rows"] is None:
        return dict(out=o)
    used = torch.arange(N, device=dev) < s["rows"].long()[:, None]
    return dict(out=s["out"].copy_(torch.where(used[:, :, None, None], o, s["out"])))


def _plain_adjust(case, s):
    B, N, V = s["logits"].shape
    dev = s["logits"].device
    z = s["logits"].float()

    def counted(ids):
        c = torch.zeros(B, V + 1, device=dev)
        if ids is not None:
            c.scatter_add_(1, torch.where(ids < 0, V, ids).long(), torch.ones(ids.shape, device=dev))
        return c[:, None, :V]

    count, prompt = counted(s["history"]), counted(s["prompt"])
    if s["tokens"] is not None:
        count = count.expand(B, N, V).clone()
        mark = torch.zeros(B, N, V, device=dev)
        mark[:, 1:].scatter_(2, s["tokens"].long()[..., None], 1.0)
        count += mark.cumsum_(1)
    theta, often, once = (s[n][:, None, None] for n in ("repetition", "frequency", "presence"))
    z = torch.where((count > 0) | (prompt > 0), torch.where(z > 0, z / theta, z * theta), z)
    z = torch.where(count > 0, z - (often * count + once), z)
    if s["bias"] is not None:
        more = torch.zeros(B, V, device=dev).scatter_(1, s["bias_ids"].long(), s["bias"])
        z += more[:, None]
    if s["allowed"] is not None:
        bit = s["allowed"][..., None] >> torch.arange(32, dtype=torch.int32, device=dev)
        z.masked_fill_(((bit & 1) == 0).view(B, N, -1)[..., :V], float("-inf"))
    return dict(logits=z.to(s["logits"].dtype))


_plain = dict(rotate=_plain_rotate, write=_plain_write, read=_plain_read, attend=_plain_attend, adjust=_plain_adjust)


# ---------------------------------------------------------------- what a pass needs


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B, N = case["B"], case.get("N", 1)
    if case["op"] == "rotate":
        cells = B * N * (case["Hq"] + case["Hk"]) * case["D"]
        return dict(bytes=2 * cells * es, flops=3 * cells)
    if case["op"] == "adjust":
        cells = B * N * case["V"]
        return dict(bytes=2 * cells * es + (cells // 8 if case["mask"] else 0), flops=2 * cells)
    H, D, before = case["H"], case["D"], _before(case)
    token = 2 * H * D
    if case["op"] == "read":
        return dict(bytes=sum(before) * token * (1 + es), flops=sum(before) * token)
    counts = _row_counts(case)
    if case["op"] == "write":
        held = sum(a % BLOCK for a in before)
        back = (held + sum(counts)) * token
        # new rows and what their blocks held, both as codes; then all of it back as values
        return dict(bytes=sum(counts) * token * (es + 1) + 2 * held * token + back * (1 + es), flops=4 * back)
    seen = kept = 0
    for a, n in zip(before, counts):
        for j in range(n):
            seen += min(a + j + 1, case["window"] or a + j + 1)
        kept += a + n - max(0, a + 1 - case["window"] if case["window"] else 0)
    return dict(bytes=kept * token + 2 * sum(counts) * case["Hq"] * D * es, flops=4 * seen * case["Hq"] * D)


# ---------------------------------------------------------------- 64 bits


def _power(e):
    """2^e in 64 bits, from e's bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """Numbers of at most 448 rounded to three bits behind the first, below 2^-6 to whole 2^-9; ties to even."""
    step = torch.full_like(x, 2.0 ** -9)
    for e in range(-5, 9):
        step = torch.where(x.abs() >= 2.0 ** e, 2.0 ** (e - 3), step)
    return torch.round(x / step) * step


def _tokens64(s, name, b, first, count):
    """Tokens first .. of request b, [count, heads, D] in 64 bits, each byte taken from its place."""
    D, page = s["case"]["D"], s["case"]["page"]
    dev = s["page_table"].device
    t, d = torch.arange(first, first + count, device=dev)[:, None, None], torch.arange(D, device=dev)
    u, e = t % BLOCK, d % 32
    if name == "k":
        place = 256 * (e // 8) + 16 * (4 * (u // 8) + u % 4) + 8 * (u // 4 % 2) + e % 8
    else:
        place = 256 * (u // 8) + 16 * (e % 16) + 8 * (e // 16) + u % 8
    codes = s[name + "_codes"].view(torch.uint8)
    head = torch.arange(codes.shape[1], device=dev)[None, :, None]
    page_of, block = s["page_table"].long()[b, t // page], t % page // BLOCK
    got = codes[page_of, head, block, d // 32, place].view(torch.float8_e4m3fn).double()
    return got * s[name + "_scale"].double()[page_of, head, block]


def _exact_rotate(case, s):
    R, N = case["R"], case["N"]
    turns = (s["kv_len"].double()[:, None] + torch.arange(N, device=s["q"].device))[..., None] * s["freqs"]
    unit = torch.polar(torch.full_like(turns, s["scale"]), turns)[:, :, None]

    def turn(x):
        y = x.double().clone()
        if case["inter"]:
            first, second = slice(0, R, 2), slice(1, R, 2)
        else:
            first, second = slice(0, R // 2), slice(R // 2, R)
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return dict(q=turn(s["q"]), k=turn(s["k"]))


def _exact_write(case, s):
    out = {}
    for name, back in zip(("k", "v"), s["out"]):
        scale, got = s[name + "_scale"].double(), back.double()
        for b, (a, n) in enumerate(zip(s["before"], s["counts"])):
            first = a // BLOCK * BLOCK
            x = torch.cat((_tokens64(s, name, b, first, a - first), s[name][b, :n].double()))
            for i in range(0, len(x), BLOCK):
                y = x[i: i + BLOCK]
                amax = y.abs().amax((0, 2))
                size = _power(torch.floor(torch.log2(amax.clamp(min=1e-30) / 448.0)) - 1)
                size = torch.where(size * 448.0 < amax, 2 * size, size)
                size = torch.where(size * 448.0 < amax, 2 * size, size)
                size = torch.where(amax > 0, size, 1.0)
                got[b, i: i + len(y)] = _e4m3(y / size[:, None]) * size[:, None]
                t = first + i
                scale[s["page_table"][b, t // case["page"]].long(), :, t % case["page"] // BLOCK] = size
        out[name], out[name + "_scale"] = got, scale
    return dict(k=out["k"], v=out["v"], k_scale=out["k_scale"], v_scale=out["v_scale"])


def _exact_read(case, s):
    got = [x.double() for x in s["out"]]
    for x, name in zip(got, ("k", "v")):
        for b, n in enumerate(s["before"]):
            x[b, :n] = _tokens64(s, name, b, 0, n)
    return dict(k=got[0], v=got[1])


def _exact_attend(case, s):
    G, D = case["Hq"] // case["H"], case["D"]
    out = s["out"].double()
    for b, (a, n) in enumerate(zip(s["before"], s["counts"])):
        first = max(0, a + 1 - case["window"]) if case["window"] else 0
        k, v = (_tokens64(s, name, b, first, a + n - first) for name in ("k", "v"))
        t = torch.arange(first, a + n, device=k.device)
        for j in range(n):
            seen = (t <= a + j) & (t > a + j - (case["window"] or a + j + 1))
            q = s["q"][b, j].double().view(case["H"], G, D)
            z = torch.matmul(q, k[seen].permute(1, 2, 0).contiguous()) / D ** 0.5
            p = torch.softmax(z, -1)
            out[b, j] = torch.matmul(p, v[seen].transpose(0, 1).contiguous()).reshape(-1, D)
    return dict(out=out)


def _exact_adjust(case, s):
    z = s["logits"].double().clone()
    B, N, V = z.shape
    for b in range(B):
        past = s["history"][b].long() if s["history"] is not None else torch.zeros(0, dtype=torch.int64, device=z.device)
        read = s["prompt"][b].long() if s["prompt"] is not None else past[:0]
        for j in range(N):
            ids = torch.cat((past, s["tokens"][b, :j].long())) if j else past
            count = torch.bincount(ids[ids >= 0], minlength=V)
            seen = count + torch.bincount(read[read >= 0], minlength=V) > 0
            theta, row = s["repetition"][b].double(), z[b, j]
            row = torch.where(seen, row * theta.pow(-torch.sign(row)), row)
            row = row - s["frequency"][b].double() * count - s["presence"][b].double() * (count > 0)
            if s["bias"] is not None:
                row[s["bias_ids"][b].long()] += s["bias"][b].double()
            if s["allowed"] is not None:
                v = torch.arange(V, device=z.device)
                row[(s["allowed"][b, j].long()[v // 32] >> (v % 32)) % 2 == 0] = float("-inf")
            z[b, j] = row
    return dict(logits=z)


def exact(case, seed):
    s = prepare(case, seed)
    forms = dict(rotate=_exact_rotate, write=_exact_write, read=_exact_read, attend=_exact_attend, adjust=_exact_adjust)
    return forms[case["op"]](case, s)
