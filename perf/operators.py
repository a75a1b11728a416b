"""The operators of a K/V cache held in 8 bits, in plain torch and as the library's calls.

The cache of ``include/gtattn.h`` (gtattn_cache): pages of `page` tokens, per
page and K/V head an e4m3 tile [page, D] and one power-of-two scale, for the
keys also the bf16 mean of the page's stored keys.  Four operators:

  slots    pages and slots for the tokens that each request adds
  append   the new tokens' keys and values into the pages, in 8 bits
  select   for each new token and K/V head, the pages that score highest
  attend   attention of the new tokens over the cache, or over those pages

and ``step``, the four one after another, as one step of a batch runs them.
With ``own`` false, `run` computes them in elementary torch operations, with
it true through ``graph_transformer_sparse_gb300``.  `exact` computes what
are numbers in 64 bits, request by request.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.bfloat16),
          "bf16_out_f32": (torch.bfloat16, torch.float32)}


def listed():
    return [
        # a batch of requests, one token each: the pages and slots of the step (latency)
        case("slots, decode", "slots", S=256, lo=1, hi=8191, page=64),
        # prompts of mixed lengths arriving at once next to requests in flight
        case("slots, prompts", "slots", S=1500, lo=0, hi=4000, add=120, page=16),
        # one token of each request into its last page (most pages partly filled)
        case("append, decode", "append", S=128, lo=1, hi=2047, Hkv=8, D=128, page=64),
        # prompts into the cache, fp32 features at the library's 8 x 64 heads
        case("append, prompts", "append", S=13, lo=0, hi=300, add=2500, Hkv=8, D=64, page=32, dtype="f32"),
        # the pages that each request's next token reads, long requests
        case("select, decode", "select", S=64, lo=9000, hi=32000, H=32, Hkv=8, D=128, page=64, n_sel=32),
        # a few tokens at a time on short ragged requests, small pages, fp32
        case("select, several", "select", S=9, lo=3, hi=3001, add=5, H=12, Hkv=4, D=64, page=16, n_sel=9, dtype="f32"),
        # the smallest call: one token of one short request, 4 x 32 heads
        case("attend, one", "attend", S=1, lo=100, hi=100, H=4, Hkv=4, D=32, page=16, dtype="f32"),
        # the ordinary one: a batch of requests of unlike lengths, grouped heads
        case("attend, decode", "attend", S=64, lo=500, hi=8191, H=32, Hkv=8, D=128, page=64),
        # one very long request alone: all its work lies along the cache
        case("attend, long", "attend", S=1, lo=262149, hi=262149, H=16, Hkv=4, D=128, page=64, dtype="bf16_out_f32"),
        # a batch of long requests, each head group on the pages chosen for it
        case("attend, selected", "attend", S=64, lo=9000, hi=32000, H=32, Hkv=8, D=128, page=64, n_sel=32),
        # a prompt's next piece against what the cache holds (arithmetic counts)
        case("attend, piece", "attend", S=3, lo=2000, hi=5000, add=509, H=16, Hkv=8, D=64, page=32),
        # a whole step: slots, append, select and attend
        case("step", "step", S=48, lo=1500, hi=6000, H=16, Hkv=8, D=64, page=32, n_sel=40),
    ]


def case(name, kind, S, lo, hi, add=1, H=8, Hkv=8, D=64, page=64, n_sel=0, dtype="bf16"):
    """S requests that hold lo..hi tokens and add 1..add each (all `add` = 1: one each)."""
    return {"name": name, "kind": kind, "S": S, "lo": lo, "hi": hi, "add": add, "H": H, "Hkv": Hkv, "D": D,
            "page": page, "n_sel": n_sel, "dtype": dtype}


def draw(rng):
    def log(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    kind = rng.choice(["slots", "append", "select", "attend", "attend", "step"])
    page, D = rng.choice([16, 32, 64]), rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f32", "bf16_out_f32"])
    S = log(1, 64)
    # tokens that the batch holds, bounded by the largest listed case's cache
    hi = log(20, max(20, min(250000, 256000000 // (S * Hkv * D))))
    add = rng.choice([1, 1, 1, log(2, 8), log(9, 400)])
    if kind == "slots":
        S, add = log(1, 1500), log(1, 120)
        hi = log(20, 8000)
    if kind in ("append", "step"):
        hi = min(hi, 6000)
    if kind in ("select", "attend") and S * add > 1600:
        add = max(1, 1600 // S)
    if kind == "attend" and S * add * H * hi > 60000000:
        add = max(1, 60000000 // (S * H * hi))
    n_sel = log(2, 40) if kind in ("select", "step") or (kind == "attend" and rng.random() < 0.4) else 0
    if n_sel and kind != "select" and S * add * Hkv * n_sel * page * D > 150000000:
        add = 1
    lo = rng.choice([0, 1, hi // 2, hi])
    return {k: v for k, v in case("", kind, S, lo, hi, add, H, Hkv, D, page, n_sel, dtype).items() if k != "name"}


def lengths(c):
    """(tokens held, tokens added) by each request: spread evenly over the case's range, in no order."""
    part = [((i + 1) * 0.6180339887498949) % 1.0 for i in range(c["S"])]
    held = [c["lo"] + int(p * (c["hi"] - c["lo"] + 1)) for p in part]
    added = [c["add"] if c["add"] == 1 or c["S"] == 1 else 1 + int(((p * 7.13) % 1.0) * c["add"]) for p in part]
    return held, added


def pages_of(tokens, page):
    return -(-tokens // page)


def work(c):
    held, added = lengths(c)
    page, D, H, Hkv, S = c["page"], c["D"], c["H"], c["Hkv"], c["S"]
    T = sum(added)
    esz, osz = (t.itemsize for t in DTYPES[c["dtype"]])
    kind, total = c["kind"], {"bytes": 0, "flops": 0}

    def put(nbytes, flops):
        total["bytes"] += nbytes
        total["flops"] += flops

    if kind in ("slots", "step"):
        fresh = sum(pages_of(h + a, page) - pages_of(h, page) for h, a in zip(held, added))
        put(4 * (4 * S + 2 * fresh + T), 4 * S + 2 * T)
    if kind in ("append", "step"):
        runs = sum(pages_of(h + a, page) - h // page for h, a in zip(held, added))
        kept = sum(h % page for h in held)   # tokens before the new ones in their first page: read for its mean
        put(2 * T * Hkv * D * (esz + 1) + kept * Hkv * D + runs * Hkv * (2 * D + 16), 6 * T * Hkv * D + kept * Hkv * D)
    if kind in ("select", "step"):
        means = sum((h + a - 1) // page for h, a in zip(held, added))
        scored = sum(a * ((h + a - 1) // page) for h, a in zip(held, added))
        put(means * (Hkv * D * 2 + 4) + T * (H * D * esz + 4 * Hkv * c["n_sel"]), 2 * scored * Hkv * D)
    if kind in ("attend", "step"):
        if c["n_sel"]:
            seen = [min(h + a, c["n_sel"] * page) for h, a in zip(held, added)]
            keys = [min(h + a, a * min(h + a, c["n_sel"] * page)) for h, a in zip(held, added)]
            pairs = sum(a * s for a, s in zip(added, seen))
        else:
            keys = [h + a for h, a in zip(held, added)]
            pairs = sum(a * h + a * (a + 1) // 2 for h, a in zip(held, added))
        put(sum(keys) * Hkv * D * 2 + sum(pages_of(k, page) for k in keys) * (8 * Hkv + 4)
            + T * H * D * (esz + osz) + 4 * T * Hkv * c["n_sel"], 4 * pairs * H * D)
    return total


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def tiles(gen, n, page, D):
    """n e4m3 tiles [page, D] as the append leaves them: normal values about a
    page's own direction, the largest near the type's largest."""
    some = min(n, 2048)
    x = torch.randn(some, page, D, generator=gen, device="cuda") + 0.7 * torch.randn(some, 1, D, generator=gen, device="cuda")
    x = x * (400.0 / x.abs().amax((1, 2), keepdim=True))
    x = x.to(torch.float8_e4m3fn)
    if some == n:
        return x
    return x.view(torch.uint8)[torch.randint(some, (n,), generator=gen, device="cuda")].view(torch.float8_e4m3fn)


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, S, page, D, H, Hkv = c["kind"], c["S"], c["page"], c["D"], c["H"], c["Hkv"]
    dt, odt = DTYPES[c["dtype"]]
    held, added = lengths(c)
    order = torch.randperm(S, generator=gen, device="cuda").tolist()
    held, added = [held[i] for i in order], [added[i] for i in order]
    T = sum(added)
    grown = [h + a for h, a in zip(held, added)]
    last = held if kind in ("slots", "step") else grown     # pages in the table before the call
    have = [pages_of(n, page) for n in last]
    P = max(pages_of(n, page) for n in grown)
    need = sum(pages_of(n, page) for n in grown)
    pages = need + 3
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dt)

    st = {"case": c, "T": T, "P": P, "held": ints(held), "add": ints(added), "longest": max(grown),
          "most": max(added), "pages": pages}
    st["length"] = ints(grown)
    st["tok_off"] = ints([0] + torch.tensor(added).cumsum(0).tolist())
    at = torch.arange(P, device="cuda")
    start = (ints(have).cumsum(0) - ints(have)).view(-1, 1)
    inside = at < ints(have).view(-1, 1)
    st["table"] = torch.where(inside, ids[(start + at).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    if kind in ("slots", "step"):
        st["free"] = ids[sum(have):].contiguous()
        st["new_length"], st["counts"] = torch.empty_like(st["held"]), torch.empty(3, dtype=torch.int32, device="cuda")
        st["new_off"] = torch.empty(S + 1, dtype=torch.int32, device="cuda")
        st["slots"] = torch.empty(T, dtype=torch.int32, device="cuda")
    if kind == "append":
        row = torch.repeat_interleave(torch.arange(S, device="cuda"), ints(added), output_size=T)
        pos = torch.arange(T, device="cuda") - st["tok_off"][row] + ints(held)[row]
        st["slots"] = (st["table"][row, pos // page] * page + pos % page).to(torch.int32)
    if kind in ("append", "attend", "step"):
        for name in ("k", "v"):
            st[name + "8"] = tiles(gen, pages * Hkv, page, D).view(pages, Hkv, page, D)
            st[name + "scale"] = torch.exp2(torch.randint(-9, -6, (pages, Hkv), generator=gen, device="cuda").float())
    if kind in ("append", "step"):
        st["kmean"] = (st["k8"].float().mean(2) * st["kscale"].unsqueeze(-1)).to(torch.bfloat16)
        st["K"], st["V"] = randn(T, Hkv, D), randn(T, Hkv, D)
    if kind == "select":
        st["kmean"] = (0.7 * torch.randn(pages, Hkv, D, generator=gen, device="cuda")).to(torch.bfloat16)
    if kind in ("select", "attend", "step"):
        st["Q"] = randn(T, H, D)
        st["scale"] = 1.0 / math.sqrt(D)
        st["out"] = torch.empty(T, H, D, dtype=odt, device="cuda")
        st["sel"] = torch.empty(T, Hkv, max(1, c["n_sel"]), dtype=torch.int32, device="cuda")
    if kind == "attend" and c["n_sel"]:
        # a choice as `select` makes it: the last visible page and others, ascending, then -1
        last_page = torch.cat([torch.arange(h, h + a) for h, a in zip(held, added)]).cuda().div(page, rounding_mode="floor")
        score = torch.rand(T, Hkv, P, generator=gen, device="cuda")
        score = torch.where(at < last_page.view(-1, 1, 1), score, -1.0)
        score = torch.where(at == last_page.view(-1, 1, 1), 2.0, score)
        n = min(P, c["n_sel"])
        top = score.topk(n, -1)
        chosen = torch.where(top.values >= 0, top.indices, P).sort(-1).values
        st["sel"].fill_(-1)
        st["sel"][..., :n] = torch.where(chosen < P, chosen, -1)
    if own:
        import graph_transformer_sparse_gb300 as gt
        st["gt"] = gt
        st["dtype"] = {"f32": gt.GTATTN_F32, "bf16": gt.GTATTN_BF16, "bf16_out_f32": gt.GTATTN_BF16_OUT_F32}[c["dtype"]]
        if kind != "slots":
            st["cache"] = gt.Cache(st.get("k8"), st.get("v8"), st.get("kscale"), st.get("vscale"), st.get("kmean"), page)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    kind = st["case"]["kind"]
    stages = ("slots", "append", "select", "attend") if kind == "step" else (kind,)
    out = {}
    if "slots" in stages:
        (own_slots if own else plain_slots)(st)
        out.update(table=st["table"], length=st["new_length"], offsets=st["new_off"], slots=st["slots"], counts=st["counts"])
    if "append" in stages:
        (own_append if own else plain_append)(st)
        out.update({k: st[k] for k in ("k8", "v8", "kscale", "vscale", "kmean")})
    if "select" in stages:
        (own_select if own else plain_select)(st)
        out.update(sel=st["sel"])
    if "attend" in stages:
        (own_attend if own else plain_attend)(st)
        out.update(out=st["out"])
    return out


def own_slots(st):
    c = st["case"]
    st["gt"].gtattn_cache_slots(st["held"], st["add"], st["table"], st["free"], st["new_length"], st["new_off"], st["slots"],
                                st["counts"], c["S"], st["P"], st["free"].numel(), st["T"], c["page"])


def own_append(st):
    st["gt"].gtattn_cache_append(st["cache"], st["K"], st["V"], st["slots"], st["T"], st["dtype"])


def own_select(st):
    c = st["case"]
    st["gt"].gtattn_cache_select(st["cache"], st["Q"], st["table"], st["length"], st["tok_off"], st["sel"], c["S"], st["T"],
                                 st["P"], c["H"], c["n_sel"], st["dtype"])


def own_attend(st):
    c = st["case"]
    st["gt"].gtattn_fwd_cache(st["cache"], st["Q"], st["table"], st["length"], st["tok_off"], st["out"], c["S"], st["T"],
                              st["P"], c["H"], st["scale"], st["dtype"], sel=st["sel"] if c["n_sel"] else None,
                              n_sel=c["n_sel"])


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def plain_slots(st):
    """Pages from the free list in request order; a token's slot is its page's id * page + its place in it."""
    page, T, table = st["case"]["page"], st["T"], st["table"]
    length, add = st["held"].long(), st["add"].long()
    grown = length + add
    have, want = (length + page - 1) // page, (grown + page - 1) // page
    ends = (want - have).cumsum(0)
    first = ends - (want - have)
    at = torch.arange(table.shape[1], device="cuda")
    fresh = (at >= have.view(-1, 1)) & (at < want.view(-1, 1))
    pick = (first.view(-1, 1) + at - have.view(-1, 1)).clamp(0, max(0, st["free"].numel() - 1))
    table.copy_(torch.where(fresh, st["free"][pick], table))
    st["new_length"].copy_(grown)
    st["new_off"][0] = 0
    st["new_off"][1:] = add.cumsum(0)
    row = torch.repeat_interleave(torch.arange(add.numel(), device="cuda"), add, output_size=T)
    pos = torch.arange(T, device="cuda") - st["new_off"][row] + length[row]
    st["slots"].copy_(table[row, pos // page] * page + pos % page)
    st["counts"].copy_(torch.stack([ends[-1], add.sum(), torch.zeros_like(ends[-1])]))


def power_scale(amax):
    """The smallest power of two 2^e with amax <= 448 * 2^e, e in [-64, 120]."""
    m, e = torch.frexp(amax)                   # amax = m 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
    e = e - 9 + (m > E4M3_MAX / 512.0).int()
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -64).clamp(-64, 120))


def plain_append(st):
    page, pages, slots = st["case"]["page"], st["pages"], st["slots"].long()
    pid, off = slots // page, slots % page
    begins = torch.ones_like(pid, dtype=torch.bool)
    begins[1:] = pid[1:] != pid[:-1]
    touched, kept = pid[begins], off[begins]                          # pages, and the tokens before the new ones
    run = begins.long().cumsum(0) - 1
    filled = torch.zeros_like(kept).scatter_reduce(0, run, off + 1, "amax")
    where = torch.arange(page, device="cuda").view(1, 1, -1, 1)
    for name in ("k", "v"):
        x8, xs, x = st[name + "8"], st[name + "scale"], st[name.upper()].float()
        amax = torch.zeros(touched.numel(), x.shape[1], device="cuda")
        amax = amax.scatter_reduce(0, run.view(-1, 1).expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        old = torch.where(kept.view(-1, 1) > 0, xs[touched], torch.zeros_like(amax))
        new = torch.maximum(old, power_scale(amax))
        tile = x8.view(torch.uint8)[touched].view(torch.float8_e4m3fn).float()
        old_part = where < kept.view(-1, 1, 1, 1)
        tile = torch.where(old_part, tile * (old / new)[..., None, None], tile)
        tile[run, :, off] = x / new[run].unsqueeze(-1)
        tile = tile.to(torch.float8_e4m3fn)
        x8.view(torch.uint8)[touched] = tile.view(torch.uint8)
        xs[touched] = new
        if name == "k":
            inside = where < filled.view(-1, 1, 1, 1)
            total = torch.where(inside, tile.float(), 0.0).sum(2) * new.unsqueeze(-1)
            st["kmean"][touched] = (total / filled.view(-1, 1, 1).float()).to(torch.bfloat16)


def rows_of(st):
    """For each new token its request and its place in the request."""
    T = st["T"]
    row = torch.repeat_interleave(torch.arange(st["case"]["S"], device="cuda"), st["add"].long(), output_size=T)
    place = torch.arange(T, device="cuda") - st["tok_off"].long()[row] + st["length"].long()[row] - st["add"].long()[row]
    return row, place


def plain_select(st):
    """The page of the token itself and, of the earlier ones, those of highest score (64 bits; ties: the first)."""
    c = st["case"]
    Hkv, P, T, n_sel = c["Hkv"], st["P"], st["T"], c["n_sel"]
    row, place = rows_of(st)
    q = st["Q"].double().view(T, Hkv, c["H"] // Hkv, c["D"]).sum(2)                    # [T, Hkv, D]
    mean = st["kmean"][st["table"].clamp(min=0).long()].double()                       # [S, P, Hkv, D]
    many = torch.zeros(c["S"], st["most"], Hkv, c["D"], dtype=torch.float64, device="cuda")
    nth = torch.arange(T, device="cuda") - st["tok_off"].long()[row]
    many[row, nth] = q
    score = torch.einsum("sahd,sphd->sahp", many, mean)[row, nth]                      # [T, Hkv, P]
    at, last = torch.arange(P, device="cuda"), (place // c["page"]).view(-1, 1, 1)
    score = torch.where(at < last, score, -math.inf)
    score = torch.where(at == last, math.inf, score)
    score, ids = torch.sort(score, dim=-1, descending=True, stable=True)
    n = min(P, n_sel)
    ids = torch.where(ids[..., :n] <= last, ids[..., :n], P).sort(-1).values
    st["sel"].fill_(-1)
    st["sel"][..., :n] = torch.where(ids < P, ids, -1)


def plain_attend(st):
    c = st["case"]
    Hkv, D, page, T, P = c["Hkv"], c["D"], c["page"], st["T"], st["P"]
    G = c["H"] // Hkv
    row, place = rows_of(st)
    table = st["table"].clamp(min=0).long()
    q = st["Q"].float().view(T, Hkv, G, D) * st["scale"]
    inner = torch.arange(page, device="cuda")
    if c["n_sel"]:
        n = min(P, c["n_sel"])
        sel = st["sel"][..., :n].long()                                                # [T, Hkv, n]
        phys = table[row.view(-1, 1, 1), sel.clamp(min=0)]
        heads = torch.arange(Hkv, device="cuda").view(1, -1, 1)
        key = gather(st["k8"], st["kscale"], phys, heads).flatten(2, 3)                # [T, Hkv, n * page, D]
        val = gather(st["v8"], st["vscale"], phys, heads).flatten(2, 3)
        pos = (sel.unsqueeze(-1) * page + inner).flatten(2)
        seen = (pos >= 0) & (pos <= place.view(-1, 1, 1)) & (sel >= 0).repeat_interleave(page, -1)
        logit = torch.einsum("thgd,thkd->thgk", q, key)
        p = softmax(logit, seen.unsqueeze(2))
        st["out"].copy_(torch.einsum("thgk,thkd->thgd", p, val).reshape(T, c["H"], D))
        return
    heads = torch.arange(Hkv, device="cuda").view(1, -1, 1)
    phys = table.unsqueeze(1)                                                          # [S, 1, P]
    key = gather(st["k8"], st["kscale"], phys, heads).flatten(2, 3)                    # [S, Hkv, P * page, D]
    val = gather(st["v8"], st["vscale"], phys, heads).flatten(2, 3)
    nth = torch.arange(T, device="cuda") - st["tok_off"].long()[row]
    many = torch.zeros(c["S"], st["most"], Hkv, G, D, device="cuda")
    many[row, nth] = q
    to = torch.full((c["S"], st["most"]), -1, device="cuda")
    to[row, nth] = place
    logit = torch.einsum("sahgd,shkd->shagk", many, key)
    seen = torch.arange(P * page, device="cuda") <= to.unsqueeze(-1)                   # [S, A, K]
    p = softmax(logit, seen[:, None, :, None])
    o = torch.einsum("shagk,shkd->sahgd", p, val)
    st["out"].copy_(o[row, nth].reshape(T, c["H"], D))


def gather(x8, scale, phys, heads):
    tile = x8.view(torch.uint8)[phys, heads].view(torch.float8_e4m3fn).float()
    return tile * scale[phys, heads][..., None, None]


def softmax(logit, seen):
    logit = torch.where(seen, logit, -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


# --------------------------------------------------------------------------
# in 64 bits, request by request
# --------------------------------------------------------------------------
def grid(x):
    """x on the e4m3 grid: 3 bits behind the leading one, ties to even, subnormals below 2^-6."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(c, seed):
    kind = c["kind"]
    if kind in ("slots", "select"):
        return None      # whole numbers
    st = prepare(c, seed)
    held, add = st["held"].tolist(), st["add"].tolist()
    first = [0]
    for a in add:
        first.append(first[-1] + a)
    each = list(zip(range(c["S"]), held, add, first))
    if c["H"] * c["D"] * sum(a * (c["n_sel"] * c["page"] if c["n_sel"] else h + a) for _, h, a, _ in each) > 4e11:
        return None
    table = st["table"].long()
    if kind == "step":
        free = st["free"].tolist()
        for i, h, a, _ in each:
            for p in range(pages_of(h, c["page"]), pages_of(h + a, c["page"])):
                table[i, p] = free.pop(0)
    cache = {n: st[n].double() for n in ("k8", "v8", "kscale", "vscale", "kmean") if n in st}
    res = {}
    if kind in ("append", "step"):
        exact_append(c, st, each, table, cache)
        res.update(cache)
    if kind in ("attend", "step"):
        sel = st["sel"]
        if kind == "step":
            sel = exact_select(c, st, each, table, cache["kmean"].float().to(torch.bfloat16).double())
        res["out"] = exact_attend(c, st, each, table, cache, sel)
    if kind == "step":   # whole numbers in the place of the others
        res = {k: res.get(k) for k in ("table", "length", "offsets", "slots", "counts", "sel", *res)}
    return res


def exact_append(c, st, each, table, cache):
    page = c["page"]
    for name in ("k", "v"):
        code, scale, x = cache[name + "8"], cache[name + "scale"], st[name.upper()].double()
        for i, h, a, t0 in each:
            for p in range(h // page, pages_of(h + a, page)):
                b, e = max(h, p * page), min(h + a, (p + 1) * page)
                f, n, pg = b - p * page, e - b, int(table[i, p])
                new = x[t0 + b - h: t0 + e - h].transpose(0, 1)                        # [Hkv, n, D]
                s = torch.exp2(torch.clamp(torch.ceil(torch.log2(new.abs().amax((1, 2)) / E4M3_MAX)), -64, 120))
                if f > 0:
                    s = torch.maximum(s, scale[pg])
                    code[pg, :, :f] = grid(code[pg, :, :f] * (scale[pg] / s)[:, None, None])
                code[pg, :, f:f + n] = grid(new / s[:, None, None])
                scale[pg] = s
                if name == "k":
                    cache["kmean"][pg] = code[pg, :, :f + n].mean(1) * s[:, None]


def exact_select(c, st, each, table, mean):
    sel = torch.full_like(st["sel"], -1)
    for i, h, a, t0 in each:
        for j in range(a):
            last = (h + j) // c["page"]
            q = st["Q"][t0 + j].double().view(c["Hkv"], -1, c["D"]).sum(1)             # [Hkv, D]
            s = (mean[table[i, :last]] * q).sum(-1)                                    # [last, Hkv]
            best = torch.argsort(-s, dim=0, stable=True)[: c["n_sel"] - 1]
            mine = torch.cat([best, torch.full_like(s[:1], last).long() if last else torch.zeros(1, c["Hkv"], device="cuda").long()])
            mine = mine.sort(0).values
            sel[t0 + j, :, : mine.shape[0]] = mine.t().int()
    return sel


def exact_attend(c, st, each, table, cache, sel):
    page, D, Hkv, G = c["page"], c["D"], c["Hkv"], c["H"] // c["Hkv"]
    out = torch.zeros(st["T"], c["H"], D, dtype=torch.float64, device="cuda")
    for i, h, a, t0 in each:
        pos = torch.arange(h + a, device="cuda")
        pg = table[i, pos // page]
        K = cache["k8"][pg, :, pos % page] * cache["kscale"][pg].unsqueeze(-1)         # [n, Hkv, D]
        V = cache["v8"][pg, :, pos % page] * cache["vscale"][pg].unsqueeze(-1)
        q = st["Q"][t0:t0 + a].double().view(a, Hkv, G, D)
        s = torch.einsum("ahgd,khd->ahgk", q, K) * st["scale"]
        hidden = (pos[None, :] > (torch.arange(a, device="cuda") + h)[:, None])[:, None, :].expand(a, Hkv, h + a)
        if c["n_sel"]:
            hidden = hidden | ~(sel[t0:t0 + a].unsqueeze(-1) == (pos // page).view(1, 1, 1, -1)).any(2)
        s = s.masked_fill(hidden.unsqueeze(2), -math.inf)
        out[t0:t0 + a] = torch.einsum("ahgk,khd->ahgd", torch.softmax(s, -1), V).reshape(a, c["H"], D)
    return out
