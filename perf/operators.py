"""The training-loss operators as measured work: top-logit packets of a teacher,
the distillation loss that reads them, and the router's balance loss.

Plain forms (elementary torch operations in 32 bits) and the library's calls
compute the same outputs from the same inputs.  Definitions:

packet   S = the k largest logits of a row (ties to the lower index, -inf never
         taken), ascending by index: fp32 values, int32 indices, the number of
         entries, and tail = log sum of exp(x / tau) over the rest of the row.
         Unused slots hold value 0 and index -1.
distill  teacher p over the packet's entries, and pt for everything else, from
         the packet and its tail; student q = softmax(s / tau), qt its mass
         outside the packet; loss = sum p log(p / q) + pt log(pt / qt).  A student
         logit of -inf takes its position out of both distributions.
balance  p = softmax of a token's router logits, c_e the ids equal to e, n tokens
         per segment, f_e = E c_e / (k n): loss = alpha sum_e f_e mean(p_e)
         + beta mean(lse^2).
"""

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
# f16 training scales its losses so that small gradients stay in the type's range
_LOSS_SCALE = {"f32": 1.0, "bf16": 1.0, "f16": 4096.0}
_DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _packet(name, T, V, k, dtype, tau=1.0, masked=0.0, pad=0):
    return {"name": name, "op": "packet", "T": T, "V": V, "k": k, "dtype": dtype, "tau": tau,
            "masked": masked, "pad": pad}


def _distill(name, way, T, V, k, dtype, tau=1.0, tail=True, masked=0.0, pad=0):
    return {"name": name, "op": "distill", "way": way, "T": T, "V": V, "k": k, "dtype": dtype,
            "tau": tau, "tail": tail, "masked": masked, "pad": pad}


def _balance(name, way, T, E, k, dtype, nseg=1, padded=False, dropped=0.0):
    return {"name": name, "op": "balance", "way": way, "T": T, "E": E, "k": k, "dtype": dtype,
            "nseg": nseg, "padded": padded, "dropped": dropped}


def listed():
    """30522 is the word vocabulary and 1000 the class count of the parameter
    sets in workloads.py; the other sizes are generic."""
    return [
        # a few tokens answered by a teacher one call at a time: latency
        _packet("packet_few_rows", 4, 30522, 64, "bf16"),
        # a teacher's forward batch over the word vocabulary
        _packet("packet_words", 8192, 30522, 64, "bf16", tau=2.0),
        # a classifier teacher: short rows, many of them
        _packet("packet_classes", 16384, 1000, 10, "f32", tau=4.0),
        # a long odd vocabulary, part of it masked, many logits kept
        _packet("packet_long_odd", 1024, 131071, 256, "f16", masked=0.05),
        # the loss of a very small step, with its gradient
        _distill("distill_step_few_rows", "both", 16, 30522, 64, "bf16", tau=2.0),
        # the ordinary training step: loss and gradient of a large batch
        _distill("distill_step_words", "both", 32768, 30522, 64, "bf16", tau=2.0),
        # validation loss over a long odd vocabulary
        _distill("distill_loss_long_odd", "loss", 4096, 131071, 128, "f16", masked=0.05),
        # the backward pass on its own, 32-bit logits in padded rows, no tail
        _distill("distill_grad_words", "grad", 8192, 30522, 32, "f32", tail=False, pad=6),
        # one small micro-batch through a small router: latency
        _balance("balance_step_small", "both", 64, 8, 2, "f32"),
        # a large batch through a wide router, loss and gradient
        _balance("balance_step_wide", "both", 131072, 256, 8, "f32"),
        # per-sequence losses of a packed batch with padding, forward only
        _balance("balance_loss_packed", "loss", 32768, 64, 6, "bf16", nseg=64, padded=True),
        # the backward pass on its own, an expert count that is no power of two, dropped ids
        _balance("balance_grad_ragged", "grad", 50001, 160, 6, "bf16", nseg=7, padded=True,
                 dropped=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packet", "distill", "distill", "balance"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "balance":
        E = _log_int(rng, 2, 512)
        T = _log_int(rng, 1, min(262144, (1 << 25) // E))
        case = _balance("", rng.choice(["both", "loss", "grad"]), T, E,
                        rng.randint(1, min(8, E)), dtype, nseg=_log_int(rng, 1, min(256, T)),
                        padded=rng.random() < 0.5, dropped=rng.choice([0.0, 0.1]))
    else:
        V = _log_int(rng, 500, 262144)
        T = _log_int(rng, 1, min(65536, (1 << 28) // V))
        masked = rng.choice([0.0, 0.0, 0.05, 0.5])
        k = _log_int(rng, 1, min(512, V // 4))
        pad = rng.choice([0, 0, 1, (-V) % 8])
        tau = rng.choice([1.0, 2.0, rng.uniform(0.5, 5.0)])
        if op == "packet":
            case = _packet("", T, V, k, dtype, tau, masked, pad)
        else:
            case = _distill("", rng.choice(["both", "loss", "grad"]), T, V, k, dtype, tau,
                            rng.random() < 0.6, masked, pad)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _rows(T, V, pad, dtype):
    """[T, V] in rows of V + pad elements."""
    return torch.empty(T, V + pad, dtype=dtype, device=_DEV)[:, :V]


def _chunk(V):
    return max(1, (1 << 26) // V)


def _vocabulary(case, gen):
    """What all rows share: a frequency prior, and the masked positions."""
    V = case["V"]
    prior = 1.5 * torch.randn(V, generator=gen, device=_DEV)
    if case["masked"]:
        gone = torch.rand(V, generator=gen, device=_DEV) < case["masked"]
        prior = torch.where(gone, torch.full_like(prior, -math.inf), prior)
    return prior


def _prepare_packet(case, seed):
    gen = _gen(seed)
    T, V, k = case["T"], case["V"], case["k"]
    prior = _vocabulary(case, gen)
    x = _rows(T, V, case["pad"], _TYPES[case["dtype"]])
    for a in range(0, T, _chunk(V)):
        b = min(T, a + _chunk(V))
        x[a:b] = 2.5 * torch.randn(b - a, V, generator=gen, device=_DEV) + prior
    return {"x": x, "values": torch.empty(T, k, device=_DEV),
            "indices": torch.empty(T, k, dtype=torch.int32, device=_DEV),
            "counts": torch.empty(T, dtype=torch.int32, device=_DEV),
            "tail": torch.empty(T, device=_DEV)}


def _prepare_distill(case, seed):
    gen = _gen(seed)
    T, V, k, tau = case["T"], case["V"], case["k"], case["tau"]
    dtype = _TYPES[case["dtype"]]
    prior = _vocabulary(case, gen)
    s = _rows(T, V, case["pad"], dtype)
    st = {"s": s, "values": torch.empty(T, k, device=_DEV),
          "indices": torch.empty(T, k, dtype=torch.int32, device=_DEV),
          "counts": torch.empty(T, dtype=torch.int32, device=_DEV), "tail": None,
          "loss": torch.empty(T, device=_DEV), "stats": torch.empty(T, 6, device=_DEV),
          "grad": None, "row_grad": None}
    tail = torch.empty(T, device=_DEV)
    for a in range(0, T, _chunk(V)):
        b = min(T, a + _chunk(V))
        x = 2.5 * torch.randn(b - a, V, generator=gen, device=_DEV) + prior
        v, i, c, t = _plain_packet(x, k, tau)
        st["values"][a:b], st["indices"][a:b], st["counts"][a:b], tail[a:b] = v, i, c, t
        s[a:b] = 0.8 * x + torch.randn(b - a, V, generator=gen, device=_DEV)
    if case["tail"]:
        st["tail"] = tail
    else:
        # packets cut to a length of their own per row
        cut = torch.randint(1, k + 1, (T,), generator=gen, device=_DEV, dtype=torch.int32)
        st["counts"] = torch.minimum(st["counts"], cut)
    # positions without a target (padding, prompts) have an empty packet
    st["counts"][torch.rand(T, generator=gen, device=_DEV) < 0.05] = 0
    if case["way"] != "loss":
        st["grad"] = _rows(T, V, case["pad"], dtype)
        weight = tau * tau * _LOSS_SCALE[case["dtype"]]
        st["row_grad"] = weight * (0.5 + torch.rand(T, generator=gen, device=_DEV))
    if case["way"] == "grad":
        for a in range(0, T, _chunk(V)):
            b = min(T, a + _chunk(V))
            st["stats"][a:b] = _plain_distill(s[a:b], st["values"][a:b], st["indices"][a:b],
                                              st["counts"][a:b], _cut(st["tail"], a, b), tau)[1]
    return st


def _cut(t, a, b):
    return None if t is None else t[a:b]


def _prepare_balance(case, seed):
    gen = _gen(seed)
    T, E, k, nseg = case["T"], case["E"], case["k"], case["nseg"]
    z = torch.randn(T, E, generator=gen, device=_DEV)
    z = (1.5 * z + torch.randn(E, generator=gen, device=_DEV)).to(_TYPES[case["dtype"]])
    ids = torch.topk(z.float(), k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        ids[torch.rand(T, k, generator=gen, device=_DEV) < case["dropped"]] = -1
    if nseg == 1:
        offs = [0, T]
    else:
        cuts = torch.randint(0, T + 1, (nseg - 1,), generator=gen, device=_DEV)
        offs = [0] + sorted(cuts.tolist()) + [T]
    mask = None
    if case["padded"]:
        mask = (torch.rand(T, generator=gen, device=_DEV) >= 0.15).to(torch.uint8)
    st = {"z": z, "ids": ids, "offs": offs, "mask": mask, "alpha": 0.01, "beta": 0.001,
          "loss": torch.empty(nseg, device=_DEV),
          "counts": torch.empty(nseg, E, dtype=torch.int32, device=_DEV),
          "tokens": torch.empty(nseg, dtype=torch.int32, device=_DEV),
          "grad": None, "seg_grad": None, "workspace": None}
    if case["way"] != "loss":
        st["grad"] = torch.empty_like(z)
        weight = T * _LOSS_SCALE[case["dtype"]] if case["dtype"] == "f16" else 1.0
        st["seg_grad"] = weight * (0.5 + torch.rand(nseg, generator=gen, device=_DEV))
    if case["way"] == "grad":
        st["counts"], st["tokens"] = _plain_counts(ids, mask, _segment_of(offs, T), nseg, E)
    if own and case["way"] != "grad":
        import error_feedback_gradient_gb300 as efg
        st["workspace"] = torch.empty(efg.balance_workspace_size(T, E, k, offs),
                                      dtype=torch.uint8, device=_DEV)
    return st


def prepare(case, seed):
    st = {"packet": _prepare_packet, "distill": _prepare_distill,
          "balance": _prepare_balance}[case["op"]](case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _lse(x):
    """log sum exp over the last axis; -inf where nothing is left."""
    m = x.amax(-1)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return torch.log(torch.exp(x - m0.unsqueeze(-1)).sum(-1)) + m0


def _plain_packet(x, k, tau):
    T, V = x.shape
    x = x.float()
    bits = x.contiguous().view(torch.int32)
    # ascending in value, then descending in index: unique 64-bit keys
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = torch.where(x == 0, torch.zeros_like(key), key).to(torch.int64)
    index = torch.arange(V, device=x.device)
    top = torch.topk(key * (1 << 31) + ((1 << 31) - 1 - index), k, dim=1).indices
    top = torch.sort(torch.where(torch.gather(x, 1, top) == -math.inf,
                                 torch.full_like(top, V), top), dim=1).values
    used = top < V
    at = torch.where(used, top, torch.zeros_like(top))
    values = torch.where(used, torch.gather(x, 1, at), torch.zeros((), device=x.device))
    rest = torch.cat([x / tau, torch.zeros(T, 1, device=x.device)], 1)
    rest.scatter_(1, top, -math.inf)
    return (values, torch.where(used, top, torch.full_like(top, -1)).to(torch.int32),
            used.sum(1).to(torch.int32), _lse(rest[:, :V]))


def _plain_distill(s, values, indices, counts, tail, tau, row_grad=None):
    """(loss, stats, grad): grad is None without row_grad.  Everything is taken
    relative to the largest student logit and the largest in the packet."""
    T, V = s.shape
    k = values.shape[1]
    zero = torch.zeros((), device=s.device)
    none = torch.full((), -math.inf, device=s.device)
    x = s.float()
    used = torch.arange(k, device=s.device) < counts.unsqueeze(1)
    slot = torch.where(used, indices.to(torch.int64), torch.full_like(indices, V).to(torch.int64))
    xs = torch.where(used, torch.gather(x, 1, slot.clamp(max=V - 1)), none)
    ts = torch.where(xs > none, values, none)
    a = x.amax(1)
    a = torch.where(a > none, a, zero)
    b = ts.amax(1)
    b = torch.where(b > none, b, zero)
    x = (x - a.unsqueeze(1)) / tau
    xs = (xs - a.unsqueeze(1)) / tau
    ts = (ts - b.unsqueeze(1)) / tau
    off = torch.cat([x, none.expand(T, 1)], 1).scatter_(1, slot, -math.inf)[:, :V]
    l_off = _lse(off)
    full = _lse(torch.stack([l_off, _lse(xs)], 1))
    lt = none.expand(T) if tail is None else torch.where(l_off > none, tail - b / tau, none)
    d = _lse(torch.stack([_lse(ts), lt], 1))
    live = d > none
    norm = torch.where(live, d, zero)
    p = torch.where(live.unsqueeze(1), torch.exp(ts - norm.unsqueeze(1)), zero)
    pt = torch.where(live, torch.exp(lt - norm), zero)
    lnorm = torch.where(live, full, zero)
    gap = norm - lnorm
    inside = torch.where(p > 0, (ts - xs) - gap.unsqueeze(1), zero)
    outside = torch.where(pt > 0, (lt - l_off) - gap, zero)
    loss = (p * inside).sum(1) + pt * outside
    stats = torch.stack([a, l_off, full, b, d, pt], 1)
    if row_grad is None:
        return loss, stats, None
    w = torch.where(live, row_grad / tau, zero)
    has_off = l_off > none
    lo = torch.where(has_off, l_off, zero)
    coef = torch.where(has_off, w * (torch.exp(lo - lnorm) - pt), zero)
    grad = coef.unsqueeze(1) * torch.exp(off - lo.unsqueeze(1))
    on = w.unsqueeze(1) * (torch.exp(xs - lnorm.unsqueeze(1)) - p)
    grad = torch.cat([grad, grad.new_zeros(T, 1)], 1).scatter_(1, slot, on)[:, :V]
    return loss, stats, grad.to(s.dtype)


def _segment_of(offs, T):
    ends = torch.tensor(offs[1:], device=_DEV)
    return torch.bucketize(torch.arange(T, device=_DEV), ends, right=True)


def _plain_counts(ids, mask, seg, nseg, E):
    T, k = ids.shape
    keep = torch.ones(T, dtype=torch.bool, device=ids.device) if mask is None else mask != 0
    tokens = torch.zeros(nseg, dtype=torch.int32, device=ids.device)
    tokens.index_add_(0, seg, keep.to(torch.int32))
    take = (ids >= 0) & keep.unsqueeze(1)
    cell = seg.unsqueeze(1) * E + torch.where(take, ids, torch.zeros_like(ids))
    counts = torch.zeros(nseg * E, dtype=torch.int32, device=ids.device)
    counts.index_add_(0, cell.reshape(-1), take.to(torch.int32).reshape(-1))
    return counts.view(nseg, E), tokens


def _plain_balance(st):
    case = st["case"]
    z, offs, mask, way = st["z"], st["offs"], st["mask"], case["way"]
    T, E, k, nseg = case["T"], case["E"], case["k"], case["nseg"]
    seg = _segment_of(offs, T)
    if way == "grad":
        counts, tokens = st["counts"], st["tokens"]
    else:
        counts, tokens = _plain_counts(st["ids"], mask, seg, nseg, E)
    keep = torch.ones(T, device=z.device) if mask is None else (mask != 0).float()
    x = z.float()
    lse = _lse(x)
    p = torch.exp(x - lse.unsqueeze(1)) * keep.unsqueeze(1)
    lse = lse * keep
    n = tokens.float().clamp(min=1)
    f = counts.float() * (E / k) / n.unsqueeze(1)
    out = {}
    if way != "grad":
        P = torch.zeros(nseg, E, device=z.device).index_add_(0, seg, p) / n.unsqueeze(1)
        Z = torch.zeros(nseg, device=z.device).index_add_(0, seg, lse * lse) / n
        out = {"loss": st["alpha"] * (f * P).sum(1) + st["beta"] * Z, "counts": counts,
               "tokens": tokens}
    if way != "loss":
        ft = f[seg]
        w = (st["seg_grad"] / n)[seg]
        inner = st["alpha"] * (ft - (ft * p).sum(1, keepdim=True))
        out["grad"] = (w.unsqueeze(1) * p * (inner + (2 * st["beta"] * lse).unsqueeze(1))).to(
            z.dtype)
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _run_own(st):
    import error_feedback_gradient_gb300 as efg
    case = st["case"]
    if case["op"] == "packet":
        efg.logits_topk(st["x"], case["k"], case["tau"], st["values"], st["indices"],
                        st["counts"], st["tail"])
        return {n: st[n] for n in ("values", "indices", "counts", "tail")}
    way = case["way"]
    if case["op"] == "distill":
        packet = (st["values"], st["indices"])
        if way == "loss":
            efg.distill_loss(st["s"], *packet, case["tau"], st["loss"], st["stats"],
                             counts=st["counts"], tail=st["tail"])
            return {"loss": st["loss"], "stats": st["stats"]}
        if way == "grad":
            efg.distill_grad(st["s"], *packet, case["tau"], st["stats"], st["grad"],
                             counts=st["counts"], row_grad=st["row_grad"])
            return {"grad": st["grad"]}
        efg.distill_loss_grad(st["s"], *packet, case["tau"], st["loss"], st["grad"],
                              counts=st["counts"], tail=st["tail"], row_grad=st["row_grad"])
        return {"loss": st["loss"], "grad": st["grad"]}
    weights = (st["alpha"], st["beta"])
    if way == "grad":
        efg.balance_grad(st["z"], case["k"], st["offs"], *weights, st["counts"], st["tokens"],
                         st["grad"], mask=st["mask"], seg_grad=st["seg_grad"])
        return {"grad": st["grad"]}
    outs = {n: st[n] for n in ("loss", "counts", "tokens")}
    if way == "loss":
        efg.balance_loss(st["z"], st["ids"], st["offs"], *weights, st["loss"], st["counts"],
                         st["tokens"], mask=st["mask"], workspace=st["workspace"])
        return outs
    efg.balance_loss_grad(st["z"], st["ids"], st["offs"], *weights, st["loss"], st["counts"],
                          st["tokens"], st["grad"], mask=st["mask"], seg_grad=st["seg_grad"],
                          workspace=st["workspace"])
    return dict(outs, grad=st["grad"])


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "packet":
        return dict(zip(("values", "indices", "counts", "tail"),
                        _plain_packet(state["x"], case["k"], case["tau"])))
    if case["op"] == "distill":
        loss, stats, grad = _plain_distill(state["s"], state["values"], state["indices"],
                                           state["counts"], state["tail"], case["tau"],
                                           state["row_grad"])
        return {"loss": {"loss": loss, "stats": stats}, "grad": {"grad": grad},
                "both": {"loss": loss, "grad": grad}}[case["way"]]
    return _plain_balance(state)


def work(case):
    T, k = case["T"], case["k"]
    size = _SIZE[case["dtype"]]
    if case["op"] == "packet":
        return {"bytes": T * case["V"] * size + T * (8 * k + 8), "flops": 4 * T * case["V"]}
    if case["op"] == "distill":
        cells = T * case["V"]
        packet = T * (8 * k + 4)
        moved = {"loss": cells * size + packet + T * 20 + (4 * T if case["tail"] else 0),
                 "grad": 2 * cells * size + packet + T * 20,
                 "both": 2 * cells * size + packet + T * 8 + (4 * T if case["tail"] else 0)}
        return {"bytes": moved[case["way"]],
                "flops": {"loss": 4, "grad": 4, "both": 7}[case["way"]] * cells}
    cells, seg = T * case["E"], case["nseg"]
    tables = 4 * seg * case["E"] + 8 * seg + (T if case["padded"] else 0)
    moved = {"loss": cells * size + 4 * T * k + tables, "grad": 2 * cells * size + tables,
             "both": 2 * cells * size + 4 * T * k + tables}
    return {"bytes": moved[case["way"]],
            "flops": {"loss": 5, "grad": 8, "both": 9}[case["way"]] * cells}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_packet(st):
    case = st["case"]
    x, k, tau = st["x"], case["k"], case["tau"]
    outs = {"values": [], "indices": [], "counts": [], "tail": []}
    for a in range(0, case["T"], _chunk(case["V"])):
        v = x[a:a + _chunk(case["V"])].double()
        order = torch.sort(v, dim=1, descending=True, stable=True)
        have = (order.values[:, :k] > -math.inf)
        counts = have.sum(1)
        picked = torch.zeros_like(v, dtype=torch.bool).scatter_(1, order.indices[:, :k], have)
        # the positions in ascending order; rows with fewer than k entries are filled up
        rank = torch.cumsum(picked, 1)
        indices = torch.searchsorted(rank, torch.arange(1, k + 1, device=v.device).expand(
            v.shape[0], k).contiguous())
        full = torch.arange(k, device=v.device) < counts.unsqueeze(1)
        got = torch.gather(v, 1, indices.clamp(max=v.shape[1] - 1))
        outs["values"].append(torch.where(full, got, torch.zeros_like(got)))
        outs["indices"].append(torch.where(full, indices, torch.full_like(indices, -1)).int())
        outs["counts"].append(counts.int())
        outs["tail"].append(torch.logsumexp((v / tau).masked_fill(picked, -math.inf), 1))
    return {n: torch.cat(t) for n, t in outs.items()}


def _exact_distill(st):
    """Both distributions written out over the row, the rest of it as one more
    outcome."""
    case = st["case"]
    T, V, tau, way = case["T"], case["V"], case["tau"], case["way"]
    step = _chunk(V)
    outs = {n: [] for n in {"loss": ("loss", "stats"), "grad": ("grad",),
                            "both": ("loss", "grad")}[way]}
    for a in range(0, T, step):
        b = min(T, a + step)
        x = st["s"][a:b].double() / tau
        picked = torch.zeros(b - a, V + 1, dtype=torch.bool, device=x.device)
        logit = torch.full((b - a, V + 1), -math.inf, dtype=torch.float64, device=x.device)
        c = st["counts"][a:b].long().unsqueeze(1)
        where = st["indices"][a:b].long()
        unused = torch.arange(where.shape[1], device=x.device) >= c
        where = where.masked_fill(unused, V)
        picked.scatter_(1, where, True)
        logit.scatter_(1, where, st["values"][a:b].double() / tau)
        picked, logit = picked[:, :V], logit[:, :V]
        logit = logit.masked_fill(~picked | (x == -math.inf), -math.inf)
        outside = x.masked_fill(picked, -math.inf)
        lse_off = torch.logsumexp(outside, 1)
        lse = torch.logsumexp(x, 1)
        lt = torch.full_like(lse, -math.inf)
        if st["tail"] is not None:
            lt = torch.where(lse_off > -math.inf, st["tail"][a:b].double(), lt)
        lse_t = torch.logaddexp(torch.logsumexp(logit, 1), lt)
        ok = (lse_t > -math.inf)
        p = torch.exp(logit - lse_t.unsqueeze(1)).masked_fill(~ok.unsqueeze(1), 0)
        pt = torch.exp(lt - lse_t).masked_fill(~ok, 0)
        q = torch.exp(x - lse.unsqueeze(1)).nan_to_num(0.0)
        qt = torch.exp(lse_off - lse).nan_to_num(0.0)
        if "loss" in outs:
            cells = torch.where(p > 0, p * ((logit - x) - (lse_t - lse).unsqueeze(1)),
                                torch.zeros_like(p))
            rest = torch.where(pt > 0, pt * ((lt - lse_off) - (lse_t - lse)),
                               torch.zeros_like(pt))
            outs["loss"].append(cells.sum(1) + rest)
        if "stats" in outs:
            # relative to the largest logits on either side
            top, top_t = x.amax(1) * tau, logit.amax(1) * tau
            top, top_t = (torch.where(v > -math.inf, v, torch.zeros_like(v))
                          for v in (top, top_t))
            outs["stats"].append(torch.stack([top, lse_off - top / tau, lse - top / tau, top_t,
                                              lse_t - top_t / tau, pt], 1))
        if "grad" in outs:
            share = torch.exp(outside - lse_off.unsqueeze(1)).nan_to_num(0.0)
            g = torch.where(picked, q - p, (qt - pt).unsqueeze(1) * share)
            w = st["row_grad"][a:b].double() / tau * ok
            outs["grad"].append(w.unsqueeze(1) * g)
    return {n: torch.cat(t) for n, t in outs.items()}


def _exact_balance(st):
    case = st["case"]
    E, k, way, offs = case["E"], case["k"], case["way"], st["offs"]
    z = st["z"].double()
    keep = torch.ones(case["T"], dtype=torch.bool, device=z.device)
    if st["mask"] is not None:
        keep = st["mask"] != 0
    loss, table, tokens, grad = [], [], [], torch.zeros_like(z)
    for s in range(case["nseg"]):
        part = torch.arange(offs[s], offs[s + 1], device=z.device)
        part = part[keep[offs[s]:offs[s + 1]]]
        n = part.numel()
        ids = st["ids"][part].long()
        c = torch.bincount(ids[ids >= 0], minlength=E)
        table.append(c.int())
        tokens.append(n)
        if n == 0:
            loss.append(torch.zeros((), dtype=torch.float64, device=z.device))
            continue
        f = c.double() * E / (k * n)
        lse = torch.logsumexp(z[part], 1)
        p = torch.softmax(z[part], 1)
        loss.append(st["alpha"] * torch.dot(f, p.mean(0)) + st["beta"] * (lse ** 2).mean())
        if way != "loss":
            back = st["alpha"] * (f - (p @ f).unsqueeze(1)) + 2 * st["beta"] * lse.unsqueeze(1)
            grad[part] = st["seg_grad"][s].double() / n * p * back
    out = {}
    if way != "grad":
        out = {"loss": torch.stack(loss), "counts": torch.stack(table),
               "tokens": torch.tensor(tokens, dtype=torch.int32, device=z.device)}
    if way != "loss":
        out["grad"] = grad
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"packet": _exact_packet, "distill": _exact_distill,
            "balance": _exact_balance}[case["op"]](st)
