"""GPU parity of tp_attn_tree and tp_attn_decode_kv8 against the fp64 oracle.

Both receive the same bf16 queries and the same cache (bf16 rows, or codes and
scales), so what differs is arithmetic.  Bound per element, with A = sum_j p_j
|v_j| from the oracle:
  - the result is rounded once to bf16: 2^-8 of its value
  - a softmax weight over the cached keys is rounded to bf16 (2^-8 of it), or
    held, times its value scale, in three E5M2 terms or in fp16 (2^-9 of it, or
    2^-22 of the largest weight times the largest value scale): 2^-8 A
  - scores are fp32 sums: 2^-17 of sum |q k| / sqrt(d) at most, and with an 8-bit
    cache the queries' two E4M3 terms are off by up to 2^-17 of the head's
    largest element.  Scores here have sum |q k| / sqrt(d) under 64, so a
    weight is off by under 2^-10 of itself from them, and its normaliser too:
    2^-9 A
  so |error| <= 2^-8 |ref| + (2^-8 + 2^-9) A.
"""
import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_linear_column_b200 as tp

pytestmark = pytest.mark.gpu

D = 128


def _parents(T, seed):
    rng = np.random.default_rng(seed)
    return [-1] + [int(rng.choice([i - 1, rng.integers(-1, i)])) for i in range(1, T)]


def _words(kind, T, seed):
    if kind == "causal":
        return None
    if kind == "tree":
        return tp.tp_tree_mask(_parents(T, seed))
    g = torch.Generator().manual_seed(seed)
    n = (T + 63) // 64
    w = torch.randint(-2 ** 62, 2 ** 62, (T, n), generator=g) * 2 + 1  # any bits, at or above T too
    if kind == "empty":  # some rows name nothing
        w[::2] = 0
        if T % 64:
            w[::2, -1] = -1 << (T % 64)  # only bits at or above T
    return w


class Case:
    def __init__(self, eight, T, past, nq, nkv, kind="tree", seed=0, q_size=1.5, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.eight, self.T, self.past, self.nq, self.nkv = eight, T, past, nq, nkv
        x = torch.randn(T, nq + 2 * nkv, D, generator=g)
        x[:, :nq] *= q_size
        self.qkv = x.to(torch.bfloat16).reshape(T, -1)
        n = past + T + extra
        k = torch.randn(nkv, n, D, generator=g) * torch.exp(0.3 * torch.randn(nkv, 1, D, generator=g))
        v = torch.randn(nkv, n, D, generator=g) * torch.exp(torch.randn(nkv, n, 1, generator=g))
        self.words = _words(kind, T, seed)
        self.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))

    def set_cache(self, k, v):
        """bf16 caches; the rows behind `past` hold NaN."""
        past = self.past
        if self.eight:
            self.cache = []
            for m in (k, v):
                codes, scale = (torch.from_numpy(a) for a in oracle.kv8_quantize(m))
                codes[:, past:], scale[:, past:] = 0x7f, float("nan")
                self.cache += [codes, scale]
        else:
            self.cache = [k.clone(), v.clone()]
            for m in self.cache:
                m[:, past:] = float("nan")

    def reference(self):
        T, past, nq, nkv = self.T, self.past, self.nq, self.nkv
        new = [self.qkv.reshape(T, -1, D)[:, nq + w * nkv:nq + (w + 1) * nkv].transpose(0, 1)
               for w in (0, 1)]
        full = []
        for w in (0, 1):
            if self.eight:
                c, s = oracle.kv8_quantize(new[w])
                old = oracle.kv8_values(self.cache[2 * w][:, :past].numpy(),
                                        self.cache[2 * w + 1][:, :past].numpy())
                full.append(np.concatenate([old, oracle.kv8_values(c, s)], 1))
            else:
                full.append(np.concatenate([self.cache[w][:, :past].double().numpy(),
                                            new[w].double().numpy()], 1))
        return oracle.attn_masked(self.qkv[:, :nq * D], full[0], full[1],
                                  oracle.tree_visible(T, self.words), nq, nkv, D)

    def run(self, dev=None, t=1, **kw):
        dev = [c.cuda() for c in self.cache] if dev is None else dev
        call = tp.tp_attn_decode_kv8 if self.eight else tp.tp_attn_tree
        mask = None if self.words is None else self.words.cuda()
        ctx = call(self.qkv.cuda(), *dev, self.past, self.nq, self.nkv, D, t, tree_mask=mask, **kw)
        return ctx, dev

    def check(self, what=""):
        ctx, dev = self.run()
        torch.cuda.synchronize()
        assert tp.tp_device_error_check() == tp.TP_OK
        ref, mag = self.reference()
        y = ctx.double().cpu().numpy()
        assert np.isfinite(y).all(), what
        err = np.abs(y - ref)
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * mag
        assert (err <= bound).all(), f"{what}: {np.max(err / np.maximum(bound, 1e-300)):.3f}"
        self.check_cache(dev)
        return ctx

    def check_cache(self, dev):
        """The new rows as tp_kv_append / tp_kv8_append write them, the rest untouched."""
        want = [c.cuda() for c in self.cache]
        (tp.tp_kv8_append if self.eight else tp.tp_kv_append)(
            self.qkv.cuda(), *want, self.past, self.nq, self.nkv, D, 1)
        for a, b in zip(dev, want):
            view = torch.uint8 if a.dtype == torch.uint8 else \
                torch.int32 if a.dtype == torch.float32 else torch.int16
            assert torch.equal(a.view(view), b.view(view))


EIGHT = pytest.mark.parametrize("eight", [False, True], ids=["bf16", "kv8"])


@EIGHT
@pytest.mark.parametrize("kind", ["causal", "tree", "any"])
@pytest.mark.parametrize("past,T", [(0, 1), (1, 1), (127, 2), (128, 1), (129, 5), (1000, 4),
                                    (300, 9), (2047, 16), (513, 17)])
def test_70b_heads(eight, past, T, kind):
    Case(eight, T, past, 64, 8, kind, seed=past + T).check((past, T, kind))


@EIGHT
@pytest.mark.parametrize("nq,nkv", [(4, 4), (2, 1), (9, 3), (28, 4), (16, 1), (10, 2), (13, 1)])
@pytest.mark.parametrize("past,T", [(0, 3), (5, 1), (260, 7), (1025, 64), (640, 65), (130, 128)])
def test_head_ratios_and_row_tiles(eight, nq, nkv, past, T):
    Case(eight, T, past, nq, nkv, "tree", seed=nq + T).check((nq, nkv, past, T))


@EIGHT
@pytest.mark.parametrize("past", [0, 1, 200])
@pytest.mark.parametrize("T", [1, 2, 64, 70, 128])
def test_rows_whose_mask_names_nothing(eight, past, T):
    ctx = Case(eight, T, past, 8, 2, "empty", seed=past + T).check((past, T))
    if past == 0:
        assert (ctx[::2] == 0).all()


@EIGHT
@pytest.mark.parametrize("nq,nkv", [(8, 1), (28, 4), (16, 16), (40, 40)])
@pytest.mark.parametrize("past,T", [(129, 1), (1024, 2), (1025, 1), (1200, 4), (1537, 8), (1793, 3),
                                    (2048, 4), (2049, 4)])
def test_caches_around_eight_and_sixteen_blocks(eight, nq, nkv, past, T):
    Case(eight, T, past, nq, nkv, "any", seed=past).check((nq, nkv, past, T))


def test_short_8_bit_caches_on_two_streams_and_replayed():
    a, b = Case(True, 4, 1500, 16, 2, "tree", seed=1), Case(True, 1, 900, 16, 2, "causal", seed=2)
    want = [c.run()[0] for c in (a, b)]
    dev = [[m.cuda() for m in c.cache] for c in (a, b)]
    qkv, mask = [c.qkv.cuda() for c in (a, b)], [a.words.cuda(), None]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate((a, b)):
            got[i].append(tp.tp_attn_decode_kv8(qkv[i], *dev[i], c.past, 16, 2, D, 1,
                                                tree_mask=mask[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = [tp.tp_attn_decode_kv8(qkv[i], *dev[i], c.past, 16, 2, D, 1, tree_mask=mask[i])
                for i, c in enumerate((a, b, a, b)) for i in [i % 2]]
    for _ in range(3):
        for o in outs:
            o.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))


@EIGHT
@pytest.mark.parametrize("T", [1, 4, 30])
def test_long_cache(eight, T):
    Case(eight, T, 20011, 16, 2, "tree", seed=T).check(T)


@EIGHT
@pytest.mark.parametrize("nq,nkv", [(20, 20), (20, 10), (15, 5), (20, 4), (28, 4), (64, 8), (16, 1)])
@pytest.mark.parametrize("past,T", [(0, 128), (1, 70), (260, 66), (1025, 127), (3000, 97)])
def test_many_causal_rows(eight, nq, nkv, past, T):
    Case(eight, T, past, nq, nkv, "causal", seed=T + nq).check((nq, nkv, past, T))


@EIGHT
@pytest.mark.parametrize("past", [0, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_reaches_only_later_rows(eight, past, bad):
    # one value element of token 66 and one key element of token 90: rows 0 .. 65 of
    # their head as they were, and no other head's
    T, nq, nkv = 100, 16, 4
    c = Case(eight, T, past, nq, nkv, "causal", seed=past)
    clean, _ = c.run()
    c.qkv.view(T, -1, D)[66, nq + nkv + 1, 3] = bad
    c.qkv.view(T, -1, D)[90, nq + 2, 5] = float("nan")
    got, _ = c.run()
    same = (got == clean).view(T, nkv, -1).all(-1).cpu()
    assert same[:66].all() and same[:, [0, 3]].all() and same[:90, 2].all()
    off = ~torch.isfinite(got.view(T, nkv, -1)).all(-1).cpu()
    assert off[66:, 1].all() and off[90:, 2].all()


WIDTHS = pytest.mark.parametrize("T", [2, 20, 50], ids=["narrow", "split", "shared"])


@EIGHT
@pytest.mark.parametrize("T", [1, 3, 12, 40])
def test_scores_that_grow_along_the_cache(eight, T):
    # every key block raises the running maximum, and the value scales grow by
    # powers of two: the accumulator is rescaled again and again
    c = Case(eight, T, 1500, 8, 1, "causal", seed=T)
    g = torch.Generator().manual_seed(T)
    ramp = torch.linspace(0.05, 3.0, c.past + T + 3)[None, :, None]
    dirn = c.qkv[:, :D].float().mean(0)
    k = ramp * (dirn / dirn.norm() * 6 + 0.3 * torch.randn(1, c.past + T + 3, D, generator=g))
    v = torch.randn(1, c.past + T + 3, D, generator=g) * \
        2.0 ** torch.linspace(-20, 20, c.past + T + 3).round()[None, :, None]
    c.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))
    c.check(T)


@EIGHT
@WIDTHS
def test_one_key_far_above_a_long_flat_rest(eight, T):
    # the first key takes e^9 times the weight of each other: small weights
    # must add up
    c = Case(eight, T, 9000, 4, 1, "causal", seed=1, q_size=1.0)
    q = torch.zeros(T, 6, D)
    q[:, :4, 0] = 4.0
    q[:, 4:] = 0.5 * torch.randn(T, 2, D, generator=torch.Generator().manual_seed(2))
    c.qkv = q.to(torch.bfloat16).reshape(T, -1)
    k = 0.01 * torch.randn(1, 9003 + T, D, generator=torch.Generator().manual_seed(3))
    k[0, 0, 0] = 9.0 * np.sqrt(D) / 4
    v = 1 + 0.1 * torch.randn(1, 9003 + T, D, generator=torch.Generator().manual_seed(4))
    c.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))
    c.check()


@EIGHT
@WIDTHS
def test_values_of_zeros_and_of_very_different_sizes(eight, T):
    c = Case(eight, T, 700, 8, 2, "tree", seed=6)
    g = torch.Generator().manual_seed(7)
    k = torch.randn(2, 703 + T, D, generator=g)
    v = torch.randn(2, 703 + T, D, generator=g)
    v[0] = 0
    v[1, :300] = 0
    v[1, 300:500] *= 1e-20
    v[1, 500:] *= 1e-18
    c.qkv.view(T, -1, D)[:, 10:] *= 0
    c.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))
    ctx = c.check()
    assert (ctx.view(T, 8, D)[:, :4] == 0).all()


@WIDTHS
def test_a_large_value_scale_under_a_small_weight_costs_the_others_little(T):
    # one key far below the rest whose value is 2^10 times as large: the rest
    # keeps 2^-22 of the largest weight times the largest scale
    c = Case(True, T, 900, 4, 1, "causal", seed=2)
    g = torch.Generator().manual_seed(5)
    q = c.qkv.view(T, 6, D)
    q[:, :4, 0] = 8.0
    k = torch.randn(1, 903 + T, D, generator=g)
    v = torch.randn(1, 903 + T, D, generator=g)
    k[0, 5, 0] = -20.0
    v[0, 5] *= 1024
    c.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))
    c.check(T)


@EIGHT
@WIDTHS
def test_infinite_and_nan_scores_in_the_cache(eight, T):
    # a key that scores -inf takes no weight wherever it stands; one that scores
    # NaN makes its head's rows NaN and no other's
    c = Case(eight, T, 300, 8, 2, "causal", seed=9)
    clean, _ = c.run()
    bad = Case(eight, T, 300, 8, 2, "causal", seed=9)
    if eight:
        bad.cache[1][0, 130] = float("nan")   # the key scale
    else:
        bad.cache[0][0, 130] = float("nan")
    ctx, _ = bad.run()
    assert torch.isnan(ctx.view(T, 8, D)[:, :4]).all()
    assert torch.equal(ctx.view(T, 8, D)[:, 4:], clean.view(T, 8, D)[:, 4:])
    if not eight:
        # every key of the first block scores -inf for head group 0: the others
        # take all the weight
        low = Case(eight, T, 300, 8, 2, "causal", seed=9)
        low.qkv.view(T, -1, D)[:, :4, 0] = 1.0
        low.cache[0][0, :128, 0] = -float("inf")
        ref, mag = low.reference()
        y = low.run()[0].double().cpu().numpy()
        assert np.isfinite(y).all()
        assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * mag).all()


@EIGHT
@pytest.mark.parametrize("past", [0, 260])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T", [9, 60])
def test_what_is_not_finite_reaches_only_the_rows_that_see_it(eight, past, bad, T):
    parents = [-1, 0, 0, 1, 1, 2, -1, 6, 3] + [8] * (T - 9)
    c = Case(eight, T, past, 8, 2, "tree", seed=past)
    c.words = tp.tp_tree_mask(parents)
    clean, _ = c.run()
    at = 2  # seen by itself and token 5
    for col in (8 * D + 3, 10 * D + 4):  # its key, its value of head 0
        c2 = Case(eight, T, past, 8, 2, "tree", seed=past)
        c2.words = c.words
        c2.qkv[at, col] = bad
        ctx, _ = c2.run()
        for i in range(T):
            if i not in (2, 5):
                assert torch.equal(ctx[i], clean[i]), (i, col)
        # the other key-value head's queries do not see it either
        assert torch.equal(ctx[:, 4 * D:], clean[:, 4 * D:])
        if bad != bad:
            assert torch.isnan(ctx[at, :4 * D]).any()


@EIGHT
def test_repeats_are_bit_identical_and_calls_do_not_share_state(eight):
    a, b = Case(eight, 33, 3000, 16, 2, "tree", seed=1), Case(eight, 33, 3000, 16, 2, "tree", seed=2)
    first, _ = a.run()
    other, _ = b.run()
    for _ in range(3):
        again, _ = a.run()
        assert torch.equal(first, again)
    assert not torch.equal(first, other)
    # split over shards: the same heads, the same bits
    assert torch.equal(a.run(t=2)[0], first)


@EIGHT
def test_on_another_stream_and_in_graphs(eight):
    c = Case(eight, 12, 1111, 8, 2, "tree", seed=5)
    want, _ = c.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = c.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    # two captured graphs, each with its own workspace, replayed in turn
    dev = [[m.cuda() for m in c.cache] for _ in range(2)]
    qkv, mask = c.qkv.cuda(), c.words.cuda()
    call = tp.tp_attn_decode_kv8 if eight else tp.tp_attn_tree
    graphs, outs = [], []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call(qkv, *dev[i], c.past, 8, 2, D, 1, tree_mask=mask))
        graphs.append(gr)
    for _ in range(3):
        for gr, o in zip(graphs, outs):
            o.zero_()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


@EIGHT
def test_calls_on_two_streams_at_once(eight):
    a, b = Case(eight, 5, 9000, 16, 2, "tree", seed=1), Case(eight, 40, 9000, 16, 2, "any", seed=2)
    want = [c.run()[0] for c in (a, b)]
    call = tp.tp_attn_decode_kv8 if eight else tp.tp_attn_tree
    dev = [[m.cuda() for m in c.cache] for c in (a, b)]
    qkv, mask = [c.qkv.cuda() for c in (a, b)], [c.words.cuda() for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate((a, b)):
            got[i].append(call(qkv[i], *dev[i], c.past, 16, 2, D, 1, tree_mask=mask[i],
                               stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@EIGHT
@pytest.mark.parametrize("T", [3, 50])
def test_steps_that_follow_each_other_see_what_the_last_one_wrote(eight, T):
    # append, attend, append, attend ... without a wait in between, under each set of
    # launch options: a kernel that starts before the last one ends must still read
    # the rows and scales that it wrote, one row a step, all in one line of scales
    nq, nkv, past, steps = 8, 2, 250, 9
    g = torch.Generator().manual_seed(4)
    new = [torch.randn(1, (nq + 2 * nkv) * D, generator=g).to(torch.bfloat16).cuda()
           for _ in range(steps)]
    c = Case(eight, T, past, nq, nkv, "any", seed=7, extra=steps + 3)
    qkv, mask = c.qkv.cuda(), c.words.cuda()
    call = tp.tp_attn_decode_kv8 if eight else tp.tp_attn_tree
    append = tp.tp_kv8_append if eight else tp.tp_kv_append

    def run(wait):
        dev, out = [m.cuda() for m in c.cache], []
        torch.cuda.synchronize()
        for i, x in enumerate(new):
            append(x, *dev, past + i, nq, nkv, D, 1)
            if wait:
                torch.cuda.synchronize()
            out.append(call(qkv, *dev, past + i + 1, nq, nkv, D, 1, tree_mask=mask))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out, dev

    prev = tp.tp_get_launch_options()
    try:
        tp.tp_set_launch_options(0)
        want, cache = run(True)
        for options in (0, tp.TP_OPT_PDL, tp.TP_OPT_PDL | tp.TP_OPT_STATIC_WEIGHTS):
            tp.tp_set_launch_options(options)
            for _ in range(5):
                got, other = run(False)
                assert all(torch.equal(x, y) for x, y in zip(got, want))
                assert all(torch.equal(x[:, :past + steps], y[:, :past + steps])
                           for x, y in zip(other, cache))
    finally:
        tp.tp_set_launch_options(prev)


@EIGHT
@pytest.mark.parametrize("T", [2, 20, 50])
def test_what_a_workspace_held_does_not_matter(eight, T):
    c = Case(eight, T, 700, 8, 2, "any", seed=5)
    want, _ = c.run()
    need = tp.tp_attn_tree_workspace_bytes(T, 700, 8, 2, D)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    got, _ = c.run(workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert (ws[need:] == 0xff).all()


@EIGHT
@pytest.mark.parametrize("T", [2, 50])
def test_offsets_past_32_bits(eight, T):
    # the last head's rows start behind 2^32 elements; the first rows of each are used
    nq, nkv, past = 24, 6, 400
    n = (1 << 32) // (5 * D) + 77
    c = Case(eight, T, past, nq, nkv, "tree", seed=8)
    small = [m.cuda() for m in c.cache]
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    want, _ = c.run(dev=small)
    big = []
    for m in c.cache:
        x = torch.empty((nkv, n) + m.shape[2:], dtype=m.dtype, device="cuda")
        x[:, :m.shape[1]] = m.cuda()
        big.append(x)
    got, _ = c.run(dev=big)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for x, y in zip(big, small):
        assert torch.equal(x[:, :past + T], y[:, :past + T])


def test_the_tree_call_without_a_mask_is_decode():
    # the same operation as tp_attn_decode: both within their rounding of it
    c = Case(False, 4, 2000, 64, 8, "causal", seed=3)
    ctx = c.check().float()
    dev = [m.cuda() for m in c.cache]
    dec = tp.tp_attn_decode(c.qkv.cuda(), *dev, c.past, 64, 8, D, 8).float()
    _, mag = c.reference()
    bound = 2.0 ** -8 * dec.abs().cpu().double() + 2 * (2.0 ** -8 + 2.0 ** -9) * torch.from_numpy(mag)
    assert ((ctx - dec).abs().cpu().double() <= bound).all()


@EIGHT
def test_a_drafted_tree_is_verified_and_its_path_kept(eight):
    """The calls as a server uses them: projection, norms and rotation in place,
    the tree over the cache, the accepted path written again in order, one more
    decoded token; against the same tokens decoded one by one."""
    nq, nkv, t, past, H = 16, 2, 2, 390, 512
    g = torch.Generator().manual_seed(9)
    w = (torch.randn((nq + 2 * nkv) * D, H, generator=g) * 0.06).to(torch.bfloat16).cuda()
    wo = (torch.randn(H, nq * D, generator=g) * 0.02).to(torch.bfloat16).cuda()
    gq, gk = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    fr = (10000.0 ** (-torch.arange(64) / 64.0)).float().cuda()
    x = torch.randn(8, H, generator=g).to(torch.bfloat16).cuda()
    parents = [-1, 0, 0, 1, 2, 4]
    path = [0, 2, 4, 5]           # accepted tokens, root to leaf
    depth = [0, 1, 1, 2, 2, 3]
    base = Case(eight, 1, past, nq, nkv, "causal", seed=4, extra=20)
    attn = tp.tp_attn_decode_kv8 if eight else tp.tp_attn_tree
    keep = tp.tp_kv8_append if eight else tp.tp_kv_append

    def project(rows, positions):
        qkv, _ = tp.tp_attn_proj_forward(rows.contiguous(), w, None,
                                         torch.zeros(rows.shape[0], nq * D, dtype=torch.bfloat16,
                                                     device="cuda"), wo, None, nq, nkv, D, t)
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        return tp.tp_qk_norm_rope(qkv, 0, nq, nkv, D, t, gq, gk, fr, pos, out=qkv)

    tree = [m.cuda() for m in base.cache]
    qkv = project(x[:6], [past + k for k in depth])
    ctx = attn(qkv, *tree, past, nq, nkv, D, t, tree_mask=tp.tp_tree_mask(parents).cuda())
    keep(qkv, *tree, past, nq, nkv, D, t, rows=torch.tensor(path, dtype=torch.int32, device="cuda"))
    last = project(x[6:7], [past + 4])
    ctx_last = attn(last, *tree, past + 4, nq, nkv, D, t)

    line = [m.cuda() for m in base.cache]
    outs = []
    for n, i in enumerate(path):
        outs.append(attn(qkv[i:i + 1].clone(), *line, past + n, nq, nkv, D, t))
    out_last = attn(last, *line, past + 4, nq, nkv, D, t)
    torch.cuda.synchronize()
    for a, b in zip(tree, line):
        end = past + 5
        assert torch.equal(a[:, :end], b[:, :end])
    # a token of the path sees the same keys either way, in another order of
    # the sums: bf16 results of magnitude A, weights rounded in one of them
    for n, i in enumerate(path):
        a, b = ctx[i].float(), outs[n][0].float()
        assert (a - b).abs().max() <= 2.0 ** -6 * b.abs().max()
    assert (ctx_last.float() - out_last.float()).abs().max() <= 2.0 ** -6 * out_last.float().abs().max()


def test_a_prompt_chunk_over_an_8_bit_cache():
    """Prefill over 8-bit caches: the cached rows read back as bf16, the chunk's
    attention, the chunk's rows written in 8 bits; then one decoded token."""
    nq, nkv, past, T = 16, 2, 200, 150
    c = Case(True, T, past, nq, nkv, "causal", seed=11, extra=10)
    dev = [m.cuda() for m in c.cache]
    k = torch.zeros(nkv, past + T, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    tp.tp_kv8_read(*dev, 0, past, 1, k_out=k, v_out=v)
    ctx = tp.tp_attn_prefill(c.qkv.cuda(), k, v, past, nq, nkv, D, 1)
    tp.tp_kv8_append(c.qkv.cuda(), *dev, past, nq, nkv, D, 1)
    full = []
    for w in (0, 1):
        old = oracle.kv8_values(c.cache[2 * w][:, :past].numpy(), c.cache[2 * w + 1][:, :past].numpy())
        new = c.qkv.double().numpy().reshape(T, -1, D)[:, nq + w * nkv:nq + (w + 1) * nkv]
        full.append(np.concatenate([old, new.transpose(1, 0, 2)], 1))
    ref, mag = oracle.attn_masked(c.qkv[:, :nq * D], *full, oracle.tree_visible(T, None), nq, nkv, D)
    # keys and values were rounded to bf16 when read back: 2^-8 of each, scores
    # of size s = sum |q k| / sqrt(d) (under 32 here) off by 2^-8 s at most
    err = np.abs(ctx.double().cpu().numpy() - ref)
    assert np.linalg.norm(err) <= 1e-2 * np.linalg.norm(ref)
    one = Case(True, 1, past + T, nq, nkv, "causal", seed=12, extra=9)
    one.cache = [m.cpu().clone() for m in dev]
    one.check()
