"""GPU parity of the 4-bit key/value cache (kv4_append, kv4_read, kv4_attention) against the fp64 oracle.

Codes and scales have to be the oracle's, byte for byte: the library takes its decisions as if the rotation
had been done in 64 bits. Attention is held, element by element, to the bound of ``oracle.kv4.attention_bound``
plus the output's rounding to bf16 (2^-8 of the value).
"""
import numpy as np
import pytest

from kv4_scene import Scene, signs_of
from oracle import hadamard as Hd
from oracle import kv4 as O

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128), (256, 256)]


def dev(x, bf16=False):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(torch.bfloat16) if bf16 else t


def host(t):
    return t.double().cpu().numpy()


# ----------------------------------------------------------------------------- append

@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_append_writes_the_oracles_bytes(lib, D, G, rotate, bf16):
    """Prompts, single tokens and nothing, in one call; every byte that holds no new token stays."""
    sc = Scene([70, 1, 33, 40, 64, 129], [37, 1, 33, 0, 1, 100], heads=3, D=D, G=G, page=64, rotate=rotate, seed=D + G)
    cache = sc.cache(lib, held=sc.before())
    lib.kv4_append(cache, dev(sc.rows(sc.k), bf16), dev(sc.rows(sc.v), bf16), *sc.where())
    lib.check_device()
    got, want = cache.data.cpu().numpy(), sc.data()
    assert np.array_equal(got, want), int((got != want).sum())


def test_append_many_rows_without_a_flip(lib):
    """2 M codes of rotated rows: near-ties are decided as in 64 bits."""
    sc = Scene([2000, 1111], [2000, 1111], heads=3, D=128, G=32, page=96, seed=4)
    cache = sc.cache(lib, held=sc.before())
    lib.kv4_append(cache, dev(sc.rows(sc.k), True), dev(sc.rows(sc.v), True), *sc.where())
    assert np.array_equal(cache.data.cpu().numpy(), sc.data())


def test_append_ties_and_hard_groups(lib):
    """Exact halves round away from zero; a group far below its row's largest value; zero, subnormal and
    overflowing scales."""
    D, G = 64, 32
    for rotate in (False, True):
        sc = Scene([40], [40], heads=1, D=D, G=G, rotate=rotate, seed=9)
        g = np.random.default_rng(5)
        x = sc.bf16(g.standard_normal((40, 1, D)))
        x[0] = 0.0
        x[1] = np.tile([7.0, 0.5, 1.5, -2.5, 3.5, -0.5, 6.5, -6.5], 8)[None]        # scale 1: halves
        x[2] = np.tile([7.0, 0.5, 1.5, -2.5, 3.5, -0.5, 6.5, -6.5], 8)[None] * 2.0 ** -26   # subnormal scale
        x[3] *= 1e-9                                                                # scale 0
        x[4, :, :32] *= 1e4                                                         # one group far larger
        x[5, :, 0] = 3e6                                                            # overflowing scale
        x[6] = 1.0                                                                  # T of a constant: one value
        x[7] = 1.0 + sc.bf16(g.standard_normal((1, D)) * 0.02)
        x = sc.bf16(x)
        sc.k = [x]
        sc.v = [x[::-1].copy()]
        with np.errstate(invalid="ignore", over="ignore"):
            sc._quantise()
        cache = sc.cache(lib, held=sc.before())
        lib.kv4_append(cache, dev(sc.rows(sc.k)), dev(sc.rows(sc.v)), *sc.where())
        assert np.array_equal(cache.data.cpu().numpy(), sc.data())


def test_append_nan_marks_its_group(lib):
    import torch
    sc = Scene([40], [40], heads=2, D=64, G=32, rotate=False)
    x = sc.rows(sc.k)
    x[3, 1, 40] = np.nan
    cache = sc.cache(lib, held=sc.before())
    lib.kv4_append(cache, dev(x), dev(sc.rows(sc.v)), *sc.where())
    k, v = (host(t) for t in lib.kv4_read(cache, *sc.where(), total=sc.T, out_dtype=torch.float32))
    bad = np.zeros(k.shape, bool)
    bad[3, 1, 32:] = True
    assert np.isnan(k[bad]).all() and np.array_equal(k[~bad], np.concatenate(sc.keys)[~bad])
    assert np.array_equal(v, np.concatenate(sc.values))


@pytest.mark.parametrize("bf16", [True, False])
def test_append_strided_views(lib, bf16):
    """Keys and values as views of one fused projection's rows, heads first, and a cache that is one layer of
    several, interleaved by page."""
    import torch
    sc = Scene([50, 20], [50, 20], heads=4, D=128, G=64, page=32)
    T, H, D = sc.T, 4, 128
    kind = torch.bfloat16 if bf16 else torch.float32
    fused = torch.full((T, 3 * H * D), 99.0, dtype=kind, device="cuda")
    k, v = fused[:, H * D:2 * H * D].view(T, H, D), fused[:, 2 * H * D:].view(T, H, D)
    k.copy_(dev(sc.rows(sc.k)))
    v.copy_(dev(sc.rows(sc.v)))
    heads_first = v.transpose(0, 1).contiguous().transpose(0, 1)
    data = dev(sc.data(sc.before()))
    layers = torch.stack([data ^ 255, data, data ^ 15], 1)
    before = layers.clone()
    cache = lib.KV4Cache(layers[:, 1], D, 64, k_plan=(p := lib.Plan.rht(D, sc.signs)), v_plan=p)
    lib.kv4_append(cache, k, heads_first, *sc.where())
    assert np.array_equal(layers[:, 1].cpu().numpy(), sc.data())
    assert torch.equal(layers[:, 0], before[:, 0]) and torch.equal(layers[:, 2], before[:, 2])
    q = sc.queries(2)
    wide = torch.randn((T, 8, 2 * D), device="cuda").to(kind)
    wide[:, :, :D] = dev(q)
    table = torch.full((2, 9), 7, dtype=torch.int32, device="cuda")
    table[:, :sc.cols] = sc.where()[0]
    got = lib.kv4_attention(wide[:, :, :D], cache, table[:, :sc.cols], *sc.where()[1:], max_new=50)
    sc.check_attention(host(got), q)


# ----------------------------------------------------------------------------- read

@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("inverse", [True, False])
def test_read(lib, D, G, inverse):
    import torch
    sc = Scene([70, 1, 33, 40, 64, 129], [37, 1, 33, 0, 64, 100], heads=3, D=D, G=G, page=64, seed=D + G)
    cache = sc.cache(lib)
    k, v = lib.kv4_read(cache, *sc.where(), total=sc.T, inverse=inverse, out_dtype=torch.float32)
    kb, vb = lib.kv4_read(cache, *sc.where(), total=sc.T, inverse=inverse)
    for got, low, held in ((k, kb, sc.keys), (v, vb, sc.values)):
        ref = sc.rows(held)
        if inverse:
            ref = sc.back(ref)
            # log2 D additions and two products, each within half a step of a value below the row's sum
            tol = (np.log2(D) + 3) * 2.0 ** -24 * np.abs(sc.rows(held)).sum(-1, keepdims=True)
            assert (np.abs(host(got) - ref) <= tol).all()
        else:
            assert np.array_equal(host(got), ref)
        assert torch.equal(got.to(torch.bfloat16), low)


def test_read_leaves_other_rows_alone(lib):
    """Rows behind the last sequence stay; new tokens at positions below zero read as zeros."""
    import torch
    sc = Scene([5, 40], [5, 2], heads=2, D=64, G=32)
    cache = sc.cache(lib)
    table, lens, _ = sc.where()
    cu = dev(np.array([0, 7, 9], np.int32))      # seven new tokens of a sequence of five
    out = tuple(torch.full((12, 2, 64), -3.0, device="cuda") for _ in range(2))
    k, v = lib.kv4_read(cache, table, lens, cu, total=12, out=out)
    for got, held in ((k, sc.keys), (v, sc.values)):
        assert (got[:2] == 0).all() and (got[9:] == -3).all()
        assert np.array_equal(host(got[2:9]), np.concatenate([held[0], held[1][38:]]))
    before = cache.data.clone()
    x = torch.zeros((12, 2, 64), device="cuda")
    x[2:7], x[7:9] = dev(sc.k[0]), dev(sc.k[1][38:])
    y = torch.zeros((12, 2, 64), device="cuda")
    y[2:7], y[7:9] = dev(sc.v[0]), dev(sc.v[1][38:])
    lib.kv4_append(cache, x, y, table, lens, cu)   # writes what is there already, and nothing else
    assert torch.equal(cache.data, before)
    lib.check_device()


# ----------------------------------------------------------------------------- attention

@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("share", [1, 4, 11])
def test_attention_single_tokens(lib, D, G, rotate, share):
    lens = [1, 2, 31, 32, 33, 16, 17, 100, 257, 0]
    sc = Scene(lens, [1] * 9 + [0], heads=2, D=D, G=G, page=64, rotate=rotate, seed=D + G + share)
    q = sc.queries(share)
    cache = sc.cache(lib)
    got = lib.kv4_attention(dev(q, True), cache, *sc.where(), max_new=1, max_len=257)
    sc.check_attention(host(got), q, what="bf16")
    got = lib.kv4_attention(dev(q), cache, *sc.where(), max_new=1, max_len=257, scale=0.07)
    sc.check_attention(host(got), q, scale=0.07, what="fp32")
    lib.check_device()


@pytest.mark.parametrize("D,G", [(64, 32), (128, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("window", [0, 1, 20, 64])
@pytest.mark.parametrize("share", [1, 3, 8])
def test_attention_new_tokens(lib, D, G, window, share):
    """Several new tokens: whole prompts, drafts, chunks whose first rows end inside a tile."""
    sc = Scene([40, 1, 150, 99, 7, 200], [40, 1, 5, 33, 0, 70], heads=2, D=D, G=G, page=32, seed=D + window)
    q = sc.queries(share)
    got = lib.kv4_attention(dev(q, True), sc.cache(lib), *sc.where(), max_new=70, max_len=200, window=window)
    sc.check_attention(host(got), q, window=window)
    lib.check_device()


@pytest.mark.parametrize("D,G", [(64, 64), (128, 32), (256, 256)])
def test_attention_without_causality(lib, D, G):
    sc = Scene([40, 1, 150], [40, 1, 5], heads=1, D=D, G=G, page=96)
    q = sc.queries(2)
    got = lib.kv4_attention(dev(q, True), sc.cache(lib), *sc.where(), max_new=40, max_len=150, causal=False)
    sc.check_attention(host(got), q, causal=False)


@pytest.mark.parametrize("max_new,max_len", [(1, 1), (3, 100), (64, 5000), (300, 1 << 20), (None, None)])
def test_attention_launch_sizes_do_not_change_what_is_computed(lib, max_new, max_len):
    sc = Scene([300, 5, 1000], [64, 5, 1], heads=2, D=128, G=32, page=32, seed=3)
    q = sc.queries(4)
    got = lib.kv4_attention(dev(q, True), sc.cache(lib), *sc.where(), max_new=max_new, max_len=max_len)
    sc.check_attention(host(got), q)


@pytest.mark.parametrize("D,G,share", [(64, 32, 4), (128, 32, 4), (128, 128, 1), (256, 64, 10)])
def test_attention_long(lib, D, G, share):
    """A length that is split over many parts, and others that leave most parts empty."""
    sc = Scene([5003, 1, 700], [1, 1, 1], heads=1, D=D, G=G, page=64, seed=11)
    q = sc.queries(share, std=2.0)
    cache = sc.cache(lib)
    where = sc.where()
    assert lib.kv4_attention_workspace(cache, 3, 3, share, max_new=1, max_len=5003) > 0
    got = lib.kv4_attention(dev(q, True), cache, *where, max_new=1, max_len=5003)
    sc.check_attention(host(got), q)
    again = lib.kv4_attention(dev(q, True), cache, *where, max_new=1, max_len=5003)
    assert np.array_equal(host(got), host(again))


@pytest.mark.parametrize("k_scale,v_scale,std", [(1e4, 1.0, 1e-4), (1e-5, 1e-5, 1e4), (1.0, 2e5, 1.0), (1.0, 6e4, 1.0),
                                                 (1.0, 1e-6, 1.0),
                                                 (0.0, 1.0, 1.0), (1.0, 0.0, 0.0), (8.0, 30.0, 8.0)])
def test_attention_magnitudes(lib, k_scale, v_scale, std):
    """Values whose scales lie at either end of binary16 (at 2e5 some overflow it: a group above 7 * 65504 =
    458528 stands for NaN), sharp and flat softmaxes, zeros."""
    sc = Scene([90, 33], [2, 33], heads=2, D=64, G=32, k_scale=k_scale, v_scale=v_scale, rotate=False, outliers=False)
    q = sc.queries(3, std=std)
    got = lib.kv4_attention(dev(q), sc.cache(lib), *sc.where(), max_new=33, max_len=90)
    assert np.isfinite(host(got)).all() or v_scale == 2e5
    sc.check_attention(host(got), q)


def test_attention_scales_apart(lib):
    """Value scales that grow by 2^12 along the sequence, and from group to group: earlier sums are rescaled."""
    sc = Scene([200], [4], heads=1, D=128, G=32, rotate=False, outliers=False)
    sc.v = [sc.bf16(sc.v[0] * 2.0 ** (np.arange(200) / 16)[:, None, None] * np.repeat(2.0 ** np.arange(0, 12, 3), 32))]
    sc._quantise()
    q = sc.queries(4, std=0.1)
    got = lib.kv4_attention(dev(q), sc.cache(lib), *sc.where(), max_new=4, max_len=200)
    sc.check_attention(host(got), q)


def test_nan_reaches_only_rows_that_see_it(lib):
    """A NaN or infinite key or value of one token: rows before it, beyond its window or of other sequences
    stay as they are, rows that see it are NaN."""
    import torch
    for which, value in ((0, np.nan), (1, np.nan), (1, np.inf)):
        sc = Scene([60, 50], [30, 20], heads=1, D=64, G=32, rotate=False)
        q = sc.queries(2)
        cache = sc.cache(lib, held=[30, 50])
        rows = [sc.rows(sc.k), sc.rows(sc.v)]
        rows[which][12, 0, 5] = value         # position 42 of the first sequence
        lib.kv4_append(cache, dev(rows[0]), dev(rows[1]), *sc.where())
        for window in (0, 7):
            got = host(lib.kv4_attention(dev(q), cache, *sc.where(), max_new=30, max_len=60, window=window))
            ref, bound = None, None
            kw = dict(scale=64 ** -0.5, window=window)
            ref = O.attention(q, sc.keys, sc.values, sc.lens, sc.cu, **kw)
            bound = O.attention_bound(q, sc.keys, sc.values, sc.lens, sc.cu, **kw)
            sees = np.zeros(sc.T, bool)
            sees[12:(12 + window if window else 30)] = True
            ok = np.abs(got - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -8
            assert ok[~sees].all()
            if which == 0:
                assert np.isnan(got[sees]).all()
            else:
                assert np.isnan(got[sees][:, :, :32]).all() and ok[sees][:, :, 32:].all()


def test_pages_outside_the_cache_are_skipped_and_reported(lib):
    import torch
    sc = Scene([150, 70], [3, 1], heads=2, D=64, G=32, page=32)
    cache = sc.cache(lib)
    table, lens, cu = sc.where()
    q = sc.queries(2)
    lib.check_device()
    for bad in (-1, sc.pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        got = lib.kv4_attention(dev(q, True), cache, t, lens, cu, max_new=3, max_len=150)
        with pytest.raises(lib.RotError) as e:
            lib.check_device()
        assert e.value.status == lib.ROT_EINVAL
        gone = np.zeros(150, bool)
        gone[64:96] = True
        sc.check_attention(host(got), q, absent=[gone, np.zeros(70, bool)])
        before = cache.data.clone()
        t = table.clone()
        t[0, 4] = bad                          # the page of the new tokens
        x = torch.ones((sc.T, 2, 64), device="cuda")
        lib.kv4_append(cache, x, x, t, lens, cu)
        with pytest.raises(lib.RotError):
            lib.check_device()
        k, v = lib.kv4_read(cache, t, lens, cu, total=sc.T, out_dtype=torch.float32)
        with pytest.raises(lib.RotError):
            lib.check_device()
        assert (k[:3] == 0).all() and (v[:3] == 0).all() and (k[3] != 0).any()
        cache.data.copy_(before)
    # lengths past the table
    got = lib.kv4_attention(dev(q, True), cache, table[:, :3], lens, cu, max_new=3, max_len=150)
    with pytest.raises(lib.RotError):
        lib.check_device()
    gone = np.zeros(150, bool)
    gone[96:] = True
    sc.check_attention(host(got), q, absent=[gone, np.zeros(70, bool)])
    lib.check_device()


def test_attention_leaves_other_rows_alone(lib):
    """Rows behind the last sequence, with and without a split length; more new tokens than tokens; no page at all."""
    import torch
    for n in (60, 4000):
        sc = Scene([n, 3, 0], [2, 3, 0], heads=1, D=64, G=32)
        cache = sc.cache(lib)
        table, lens, cu = sc.where()
        q = np.concatenate([sc.queries(2), np.ones((4, 2, 64))])
        out = torch.full((9, 2, 64), -3.0, dtype=torch.bfloat16, device="cuda")
        lib.kv4_attention(dev(q, True), cache, table, lens, cu, max_new=3, max_len=n, out=out)
        sc.check_attention(host(out[:5]), q[:5])
        assert (out[5:] == -3).all()
        # the first two of five new tokens of a sequence of three stand before its beginning
        cu2 = dev(np.array([0, 2, 7, 7], np.int32))
        got = lib.kv4_attention(dev(np.concatenate([q[:2], q[:2], q[2:5]]), True), cache, table, lens, cu2, max_new=5, max_len=n)
        assert (got[2:4] == 0).all() and torch.equal(got[4:7], out[2:5])
    empty = lib.kv4_attention(dev(q[:3], True), cache, torch.zeros((3, 0), dtype=torch.int32, device="cuda"),
                              torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert (empty == 0).all()
    lib.check_device()


def test_cache_beyond_4_gib(lib):
    """Pages past 32-bit byte offsets."""
    import torch
    sc = Scene([40], [40], heads=2, D=256, G=32, page=32, seed=2)
    pages = (5 << 30) // (2 * sc.tb)
    cache = lib.KV4Cache.empty(pages, 32, 2, 256, 32, k_plan=(p := lib.Plan.rht(256, sc.signs)), v_plan=p)
    table = dev(np.array([[pages - 1, pages // 2 + 7]], np.int32))
    _, lens, cu = sc.where()
    lib.kv4_append(cache, dev(sc.k[0]), dev(sc.v[0]), table, lens, cu)
    k, _ = lib.kv4_read(cache, table, lens, cu, total=40, out_dtype=torch.float32)
    assert np.array_equal(host(k), sc.keys[0])
    q = sc.queries(2)
    got = lib.kv4_attention(dev(q), cache, table, lens, cu, max_new=40, max_len=40)
    sc.check_attention(host(got), q)
    lib.check_device()


# ----------------------------------------------------------------------------- streams, graphs, a run together

def test_on_another_stream(lib):
    import torch
    sc = Scene([3000, 40], [1, 1], heads=2, D=128, G=32)
    side = torch.cuda.Stream()
    q, where = dev(sc.queries(4), True), sc.where()
    cache = sc.cache(lib, held=sc.before())
    k, v = dev(sc.rows(sc.k)), dev(sc.rows(sc.v))
    side.wait_stream(torch.cuda.current_stream())
    lib.kv4_append(cache, k, v, *where, stream=side)
    got = lib.kv4_attention(q, cache, *where, max_new=1, max_len=3000, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        same = lib.kv4_attention(q, cache, *where, max_new=1, max_len=3000)
    side.synchronize()
    sc.check_attention(host(got), sc.queries(4))
    assert torch.equal(got, same)


def test_captured_decode_steps_follow_the_lengths(lib):
    """A decoding step (append, attention) captured once and replayed while lens grows on the device; two
    graphs with a workspace of their own, replayed on two streams at once."""
    import torch
    n0, steps = 1500, 40
    scenes = [Scene([n0 + steps, 70 + steps], [1, 1], heads=2, D=64, G=32, page=32, seed=s) for s in (0, 1)]
    runs = []
    for sc in scenes:
        cache = sc.cache(lib, held=sc.lens - steps)
        table = dev(sc.table)
        lens = dev(sc.lens - steps)
        k, v = (torch.zeros((2, 2, 64), device="cuda") for _ in range(2))
        q = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        ws = torch.zeros(lib.kv4_attention_workspace(cache, 2, 2, 8, max_new=1, max_len=2048), dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0

        def step():
            lens.add_(1)
            lib.kv4_append(cache, k, v, table, lens)
            lib.kv4_attention(q, cache, table, lens, max_new=1, max_len=2048, out=out, workspace=ws)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):   # once eagerly, as warm-up; its token is written again below
            step()
            lens.sub_(1)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((graph, s, k, v, q, out, ws, cache, lens, table))   # (all that the graph reads stays alive)
    for i in range(steps):
        queries = []
        for sc, (graph, s, k, v, q, out, *_) in zip(scenes, runs):
            at = [int(n) - steps + i for n in sc.lens]
            k.copy_(dev(np.stack([sc.k[b][at[b]] for b in (0, 1)])))
            v.copy_(dev(np.stack([sc.v[b][at[b]] for b in (0, 1)])))
            x = sc.queries(4, seed=i)
            q.copy_(dev(x))
            queries.append(x)
        torch.cuda.synchronize()
        for graph, s, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        if i % 13 == 0 or i == steps - 1:
            for sc, run, x in zip(scenes, runs, queries):
                now = Scene.__new__(Scene)
                now.__dict__.update(sc.__dict__)
                now.lens = sc.lens - steps + i + 1
                now.keys = [y[:n] for y, n in zip(sc.keys, now.lens)]
                now.values = [y[:n] for y, n in zip(sc.values, now.lens)]
                now.check_attention(host(run[5]), x, what=i)
    for sc, run in zip(scenes, runs):
        assert np.array_equal(run[7].data.cpu().numpy(), sc.data())
    lib.check_device()


def test_a_layer_from_activations_to_output(lib):
    """As a user runs them: a W4A4 projection to queries, keys and values, the cache written, attention over it
    and the W4A4 output projection; a prompt, then tokens one by one. The same tokens written and attended in
    one call give the same cache, and attention within both calls' bounds."""
    import torch
    import workloads as W
    H, share, D, G, K, steps = 2, 2, 64, 32, 256, 5
    Hq = H * share
    g = W.rng(3)
    plan = lib.Plan.rht(K, W.signs(g, K))
    head = lib.Plan.rht(D, signs_of(D))
    oplan = lib.Plan.rht(Hq * D, W.signs(g, Hq * D))
    weight = lambda n, k, pl: lib.rot_quant(dev(g.standard_normal((n, k)).astype(np.float32) * 0.08), pl, 4, 64)
    wqkv, wo = weight((Hq + 2 * H) * D, K, plan), weight(K, Hq * D, oplan)
    lens_all = [45 + steps, 20 + steps]
    x = [dev(g.standard_normal((n, K)), True) for n in lens_all]
    table = dev(np.array([[3, 0], [2, 4]], np.int32))

    def layer(cache, rows, lens, cu, max_new):
        qkv = lib.w4a4_linear_act(rows, plan, *wqkv, 64, out_dtype=torch.bfloat16).view(-1, Hq + 2 * H, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        lib.kv4_append(cache, k, v, table, lens, cu)
        o = lib.kv4_attention(q, cache, table, lens, cu, max_new=max_new, max_len=64)
        return o, lib.w4a4_linear_act(o.view(-1, Hq * D), oplan, *wo, 64), (q, k, v)

    def fresh():
        c = lib.KV4Cache.empty(5, 32, H, D, G, k_plan=head, v_plan=head)
        c.data.fill_(0x7F)
        return c
    one, many = fresh(), fresh()
    i32 = lambda a: dev(np.array(a, np.int32))
    o_all, y_all, (q_all, k_all, v_all) = layer(one, torch.cat(x), i32(lens_all), i32([0, lens_all[0], sum(lens_all)]), max(lens_all))
    got = [[], []]
    n = [l - steps for l in lens_all]
    o, y, _ = layer(many, torch.cat([a[:m] for a, m in zip(x, n)]), i32(n), i32([0, n[0], sum(n)]), max(n))
    got[0].append(o[:n[0]]), got[1].append(o[n[0]:])
    for s in range(steps):
        o, y, _ = layer(many, torch.stack([a[m + s] for a, m in zip(x, n)]), i32([m + s + 1 for m in n]), None, 1)
        got[0].append(o[:1]), got[1].append(o[1:])
    # the projections of one row and of many differ in the order of their fp32 sums only; where a row of the
    # two runs is the same, so are its codes
    assert y.isfinite().all() and y_all.isfinite().all()
    sc = Scene.__new__(Scene)
    sc.__dict__.update(D=D, G=G, heads=H, rotate=True, signs=signs_of(D), lens=np.array(lens_all), new=np.array(lens_all),
                       cu=np.array([0, lens_all[0], sum(lens_all)]), T=sum(lens_all))
    split = lambda t: [host(t[:lens_all[0]]), host(t[lens_all[0]:])]
    sc.k, sc.v = split(k_all), split(v_all)
    sc._quantise()
    sc.check_attention(host(o_all), host(q_all), what="one call")
    for cache in (one, many):
        k, v = lib.kv4_read(cache, table, i32(lens_all), i32(sc.cu), total=sc.T, out_dtype=torch.float32)
        assert np.isfinite(host(k)).all() and np.isfinite(host(v)).all()
    k, v = lib.kv4_read(one, table, i32(lens_all), i32(sc.cu), total=sc.T, out_dtype=torch.float32)
    assert np.array_equal(host(k), np.concatenate(sc.keys)) and np.array_equal(host(v), np.concatenate(sc.values))
    # token by token: attention over what that run's own cache holds
    k, v = lib.kv4_read(many, table, i32(lens_all), i32(sc.cu), total=sc.T, out_dtype=torch.float32)
    sc.keys, sc.values = split(k), split(v)
    a, b = torch.cat(got[0] + got[1]), o_all
    rel = (a.float() - b.float()).norm() / b.float().norm()
    assert rel < 0.05, float(rel)
    lib.check_device()


# ----------------------------------------------------------------------------- many rows to a key head

@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("window", [0, 90])
def test_attention_many_rows(lib, D, G, rotate, window):
    """Row tiles that are full, half empty and missing, sequences from one token on, several row chunks and steps."""
    sc = Scene([700, 1, 129, 40, 300], [300, 1, 128, 40, 0], heads=1, D=D, G=G, page=64, rotate=rotate, seed=D + G + window)
    q = sc.queries(2)
    got = lib.kv4_attention(dev(q, True), sc.cache(lib), *sc.where(), max_new=300, max_len=700, window=window)
    sc.check_attention(host(got), q, window=window)
    got = lib.kv4_attention(dev(q), sc.cache(lib), *sc.where(), max_new=300, max_len=700, window=window, scale=-0.05)
    sc.check_attention(host(got), q, window=window, scale=-0.05)
    lib.check_device()


@pytest.mark.parametrize("k_scale,v_scale,std", [(1e4, 1.0, 1e-4), (1e-5, 1e-5, 1e4), (1.0, 6e4, 1.0), (1.0, 2e5, 1.0),
                                                 (1.0, 1e-6, 1.0), (0.0, 1.0, 1.0), (1.0, 0.0, 0.0), (8.0, 30.0, 8.0)])
def test_attention_many_rows_magnitudes(lib, k_scale, v_scale, std):
    """As test_attention_magnitudes (at 2e5 some groups overflow their scale and stand for NaN)."""
    sc = Scene([150, 200], [150, 60], heads=1, D=64, G=32, k_scale=k_scale, v_scale=v_scale, rotate=False, outliers=False)
    q = sc.queries(3, std=std)
    got = lib.kv4_attention(dev(q), sc.cache(lib), *sc.where(), max_new=150, max_len=200)
    sc.check_attention(host(got), q)


def test_attention_many_rows_scales_apart(lib):
    """Value scales that grow by 2^12 along the sequence, and from group to group."""
    sc = Scene([400], [130], heads=1, D=128, G=32, rotate=False, outliers=False)
    sc.v = [sc.bf16(sc.v[0] * 2.0 ** (np.arange(400) / 32)[:, None, None] * np.repeat(2.0 ** np.arange(0, 12, 3), 32))]
    sc._quantise()
    q = sc.queries(2, std=0.1)
    got = lib.kv4_attention(dev(q), sc.cache(lib), *sc.where(), max_new=130, max_len=400)
    sc.check_attention(host(got), q)


def test_many_rows_nan_reaches_only_rows_that_see_it(lib):
    for which, value in ((0, np.nan), (1, np.nan), (1, np.inf)):
        sc = Scene([300], [200], heads=1, D=64, G=32, rotate=False)
        q = sc.queries(2)
        cache = sc.cache(lib, held=[100])
        rows = [sc.rows(sc.k), sc.rows(sc.v)]
        rows[which][72, 0, 5] = value         # position 172
        lib.kv4_append(cache, dev(rows[0]), dev(rows[1]), *sc.where())
        for window in (0, 50):
            got = host(lib.kv4_attention(dev(q), cache, *sc.where(), max_new=200, max_len=300, window=window))
            kw = dict(scale=64 ** -0.5, window=window)
            ref = O.attention(q, sc.keys, sc.values, sc.lens, sc.cu, **kw)
            bound = O.attention_bound(q, sc.keys, sc.values, sc.lens, sc.cu, **kw)
            sees = np.zeros(sc.T, bool)
            sees[72:(72 + window if window else 200)] = True
            ok = np.abs(got - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -8
            assert ok[~sees].all()
            if which == 0:
                assert np.isnan(got[sees]).all()
            else:
                assert np.isnan(got[sees][:, :, :32]).all() and ok[sees][:, :, 32:].all()


def test_many_rows_pages_outside_the_cache(lib):
    sc = Scene([600, 70], [150, 70], heads=2, D=64, G=32, page=32)
    cache = sc.cache(lib)
    table, lens, cu = sc.where()
    q = sc.queries(2)
    lib.check_device()
    t = table.clone()
    t[0, 2], t[0, 9], t[1, 1] = -1, sc.pages, 2 ** 31 - 1
    got = lib.kv4_attention(dev(q, True), cache, t, lens, cu, max_new=150, max_len=600)
    with pytest.raises(lib.RotError) as e:
        lib.check_device()
    assert e.value.status == lib.ROT_EINVAL
    gone = [np.zeros(600, bool), np.zeros(70, bool)]
    gone[0][64:96] = gone[0][288:320] = gone[1][32:64] = True
    sc.check_attention(host(got), q, absent=gone)
    lib.check_device()


def test_many_rows_split_and_left_alone(lib):
    """A length split over CTAs; launch sizes that name too few rows; rows behind the last sequence."""
    import torch
    sc = Scene([3000, 70], [70, 20], heads=1, D=128, G=32, page=64)
    cache = sc.cache(lib)
    table, lens, cu = sc.where()
    q = np.concatenate([sc.queries(2), np.ones((5, 2, 128))])
    out = torch.full((95, 2, 128), -3.0, dtype=torch.bfloat16, device="cuda")
    assert lib.kv4_attention_workspace(cache, 2, 95, 2, max_new=70, max_len=3000) > 0
    lib.kv4_attention(dev(q, True), cache, table, lens, cu, max_new=70, max_len=3000, out=out)
    sc.check_attention(host(out[:90]), q[:90])
    assert (out[90:] == -3).all()
    sc = Scene([900, 70], [800, 20], heads=1, D=64, G=64, page=64)
    q = sc.queries(1)
    got = lib.kv4_attention(dev(q, True), sc.cache(lib), *sc.where(), max_new=70, max_len=100)
    sc.check_attention(host(got), q)
    got = lib.kv4_attention(dev(q, True), sc.cache(lib), *sc.where(), max_new=800, max_len=900, causal=False)
    sc.check_attention(host(got), q, causal=False)
    lib.check_device()


# ----------------------------------------------------------------------------- refusals of the binding

def test_binding_refusals(lib):
    """What is not of the documented type, shape, layout or device is refused before any launch."""
    import torch
    sc = Scene([40, 33], [2, 1], heads=2, D=64, G=32)
    cache = sc.cache(lib)
    table, lens, cu = sc.where()
    q, k = dev(sc.queries(2)), dev(sc.rows(sc.k))
    ok = dict(q=q, table=table, lens=lens, cu=cu)
    bad = [dict(table=table.long()), dict(table=table[:1]), dict(table=table[0]), dict(table=table.t().contiguous().t()),
           dict(table=table.cpu()), dict(table=None), dict(lens=lens.float()), dict(lens=lens[:, None]), dict(lens=lens[:1]),
           dict(lens=lens.cpu()), dict(lens=[40, 33]), dict(cu=cu[:2]), dict(cu=cu.long()), dict(cu=cu.cpu()), dict(cu=None),
           dict(cu=torch.zeros(6, dtype=torch.int32, device="cuda")[::2]), dict(q=q[:, :, :32]), dict(q=q[0]),
           dict(q=q.half()), dict(q=q.cpu()), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=q[:, :3]),
           dict(q=torch.zeros(3 * 4 * 64 + 1, device="cuda")[1:].view(3, 4, 64)), dict(q=None)]
    for b in bad:
        a = ok | b
        with pytest.raises(lib.RotError) as e:
            lib.kv4_attention(a["q"], cache, a["table"], a["lens"], a["cu"], max_new=2, max_len=40)
        assert e.value.status == lib.ROT_EINVAL, b
    for kw in (dict(out=torch.empty((3, 4, 64), device="cuda")), dict(out=torch.empty((3, 4, 65), dtype=torch.bfloat16, device="cuda")),
               dict(max_len=1 << 20, max_new=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
               dict(workspace=torch.empty(16, device="cuda")), dict(window=-1), dict(window=3, causal=False),
               dict(scale=float("nan")), dict(max_new=-1), dict(max_len=-1)):
        with pytest.raises(lib.RotError):
            lib.kv4_attention(q, cache, table, lens, cu, **(dict(max_new=2, max_len=40) | kw))
    for kk, vv in ((k, k.bfloat16()), (k, k[:2]), (k[:, :1], k[:, :1]), (k.half(), k.half()), (k, None)):
        with pytest.raises(lib.RotError):
            lib.kv4_append(cache, kk, vv, table, lens, cu)
    for kw in (dict(total=3, cu=None), dict(out_dtype=torch.float16), dict(out=(k, k.bfloat16())), dict(out=(k[:2], k))):
        with pytest.raises(lib.RotError):
            lib.kv4_read(cache, table, lens, **(dict(total=3, cu=cu) | kw))
    sc.plan.close()
    with pytest.raises(lib.RotError):
        lib.kv4_attention(q, cache, table, lens, cu, max_new=2, max_len=40)
    harp = lib.Plan(64, [4, 16], stage_params=[np.linalg.qr(np.random.default_rng(0).standard_normal((4, 4)))[0][None], None])
    with pytest.raises(lib.RotError) as e:     # not one Walsh-Hadamard transform
        lib.kv4_append(lib.KV4Cache(cache.data, 64, 32, k_plan=harp), k, k, table, lens, cu)
    assert e.value.status == lib.ROT_EUNSUPPORTED
    with pytest.raises(lib.RotError):
        lib.KV4Cache(cache.data, 64, 32, k_plan=lib.Plan.rht(128))
    lib.check_device()


@pytest.mark.parametrize("new,share", [(1, 4), (6, 2), (40, 8)])
@pytest.mark.parametrize("n", [400, 1000])
def test_pages_before_a_window_may_be_gone(lib, new, share, n):
    """Table entries of pages that no row's window reaches are not looked at, by either kernel."""
    sc = Scene([n, 333], [new, 1], heads=1, D=128, G=64, page=32)
    cache = sc.cache(lib)
    table, lens, cu = sc.where()
    q = sc.queries(share)
    w = 100
    lib.check_device()
    t = table.clone()
    for b, m in ((0, new), (1, 1)):
        t[b, :max(0, int(sc.lens[b]) - m + 1 - w) // 32] = -1
    got = lib.kv4_attention(dev(q, True), cache, t, lens, cu, max_new=new, max_len=n, window=w)
    sc.check_attention(host(got), q, window=w)
    lib.check_device()


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("which", ["keys", "values", "both apart", "no signs"])
def test_rotations_of_keys_and_values_are_apart(lib, rows, which):
    """Keys and values each unrotated, rotated by plans of their own, or by a plan without signs."""
    import torch
    D, G, n = 64, 32, 90
    g = np.random.default_rng(len(which))
    sk, sv = {"keys": (signs_of(D), None), "values": (None, signs_of(D)), "both apart": (signs_of(D), signs_of(D, 5)),
              "no signs": (np.ones(D, np.int8), np.ones(D, np.int8))}[which]
    plan = lambda s: None if s is None else lib.Plan.rht(D, None if which == "no signs" else s)
    cache = lib.KV4Cache.empty(4, 32, 1, D, G, k_plan=plan(sk), v_plan=plan(sv))
    k, v = (Scene.bf16(g.standard_normal((n, 1, D)) * np.where(g.random(D) < 0.1, 9.0, 1.0)) for _ in range(2))
    i32 = lambda a: dev(np.array(a, np.int32))
    table = i32([[2, 0, 3]])
    lib.kv4_append(cache, dev(k), dev(v), table, i32([n]), i32([0, n]))
    held = []
    for x, s in ((k, sk), (v, sv)):
        codes, scale = O.quantise_rows(x[:, 0], G, s, s is not None)
        held.append(O.dequantise(codes, scale, G)[:, None])
    got = lib.kv4_read(cache, table, i32([n]), i32([0, n]), total=n, out_dtype=torch.float32)
    assert np.array_equal(host(got[0]), held[0]) and np.array_equal(host(got[1]), held[1])
    q = Scene.bf16(g.standard_normal((rows, 1, D)))
    turn = lambda x, s, inv: x if s is None else Hd.rht_apply(x.reshape(-1, D), s, inverse=inv).reshape(x.shape)
    cu = [0, rows]
    kw = dict(scale=D ** -0.5)
    qr = turn(np.float64(q), sk, False)
    ref = turn(O.attention(qr, [held[0]], [held[1]], [n], cu, **kw), sv, True)
    bound = O.attention_bound(qr, [held[0]], [held[1]], [n], cu, unrotate=sv is not None, **kw)
    out = host(lib.kv4_attention(dev(q), cache, table, i32([n]), i32(cu), max_new=rows, max_len=n))
    assert (np.abs(out - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -8).all()
    assert np.linalg.norm(out - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    k_back, v_back = (host(x) for x in lib.kv4_read(cache, table, i32([n]), i32([0, n]), total=n, inverse=True, out_dtype=torch.float32))
    for back, x, s in ((k_back, held[0], sk), (v_back, held[1], sv)):
        assert np.abs(back - turn(x, s, True)).max() <= 9 * 2.0 ** -24 * np.abs(x).sum(-1).max()


@pytest.mark.parametrize("new", [1, 90])
def test_bounded_waits_give_up_then_recover(lib, new):
    """No cache tile is copied (the testing hook): the waits run out after 20 ms, the launch ends and is reported
    once, and the next call is right. By both kernels."""
    sc = Scene([200], [new], heads=1, D=64, G=32)
    cache = sc.cache(lib)
    q = sc.queries(2)
    lib.check_device()
    lib.test_inject(lib.ROT_TEST_KV4_LOADS, 20_000_000)
    try:
        lib.kv4_attention(dev(q), cache, *sc.where(), max_new=new, max_len=200)
        with pytest.raises(lib.RotError) as e:
            lib.check_device()
        assert e.value.status == lib.ROT_ETIMEOUT
    finally:
        lib.test_inject(lib.ROT_TEST_NONE, 0)
    lib.check_device()
    got = lib.kv4_attention(dev(q), cache, *sc.where(), max_new=new, max_len=200)
    sc.check_attention(host(got), q)
    lib.check_device()


@pytest.mark.parametrize("B", [1, 30, 31, 32, 33, 70])
def test_places_of_few_and_many_sequences(lib, B):
    """Uneven and empty sequences, the first and last of them empty where there are several, before and behind the
    number whose starts a warp looks at in one go; rows behind the last one stay."""
    import torch
    new = [(5 * b) % 7 * (0 < b < B - 1) if B > 1 else 19 for b in range(B)]
    sc = Scene([n + b % 40 for b, n in enumerate(new)], new, heads=3, D=64, G=32, seed=B)
    cache = sc.cache(lib, sc.before())
    behind = 21
    k, v = (torch.cat([dev(sc.rows(x)), torch.full((behind, 3, 64), float("nan"), device="cuda")]) for x in (sc.k, sc.v))
    lib.kv4_append(cache, k, v, *sc.where())
    assert np.array_equal(cache.data.cpu().numpy(), sc.data())
    out = tuple(torch.full((sc.T + behind, 3, 64), -3.0, device="cuda") for _ in range(2))
    lib.kv4_read(cache, *sc.where(), total=sc.T + behind, out=out)
    for got, held in zip(out, (sc.keys, sc.values)):
        assert np.array_equal(host(got[:sc.T]), sc.rows(held)) and (got[sc.T:] == -3).all()
    lib.check_device()


def test_a_bad_scale_reads_into_its_own_row(lib):
    """Tokens are transformed sixteen at a time: an infinite or NaN scale reaches no other token's values."""
    import torch
    sc = Scene([48], [48], heads=2, D=128, G=32)
    cache = sc.cache(lib)
    clean = lib.kv4_read(cache, *sc.where(), total=48, inverse=True)
    bad = [3, 11, 30]
    x = [dev(sc.rows(r)) for r in (sc.k, sc.v)]
    for r in x:
        r[bad[0], :, 40] = float("nan")
        r[bad[1], :, 7] = float("inf")
        r[bad[2], 1] = 1e9
    lib.kv4_append(cache, *x, *sc.where())
    got = lib.kv4_read(cache, *sc.where(), total=48, inverse=True)
    keep = torch.ones((48, 2), dtype=torch.bool, device="cuda")
    keep[bad[0]], keep[bad[1]], keep[bad[2], 1] = False, False, False
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(a[~keep]).all(-1).any()
