"""The attention step at the edges of what its entry points take: value scales at the ends of
their range, values that do not depend on the weights, and rows that stand at odd addresses."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_token_amd as fp8
from fp8_w8a8_quantized_token_amd import _lib
from oracle import e4m3
from tests._helpers import bf16_out_to_f64, require_gpu
from tests.test_gpu_kv_cache import attend, make, on_gpu, reference

pytestmark = pytest.mark.gpu

# (rows, head dimension): tiles of 16 rows, of 128, and of 256
FORMS = [(1, 64), (1, 128), (300, 64), (300, 128)]


def code_of(x):
    return int(e4m3.encode(np.array([x], np.float32))[0])


def assert_weighted(got, ref, weight, slack=0.0, lost=0.0):
    """One rounding of each weight, shared by the sum that divides them, moves an output by up to
    2^-8 sum_j p_j |v_j - out| <= 2^-7 weight, its own rounding by 2^-8 of it; exponents of up to
    2^7 in fp32 are off by less than 2^-15. `slack`: what the scores are off by besides."""
    err = np.abs(bf16_out_to_f64(got) - ref)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -15 + slack) * weight + lost
    assert np.all(err <= bound), float(np.nanmax(err / (bound + 1e-300)))


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("count,dim", FORMS)
@pytest.mark.parametrize("lead,early,late", [(39, -100, -100), (30, -100, -100), (38, -90, -90), (39, -60, -60),
                                             (130, 0, -100), (39, -100, 0), (100, 20, -80), (20, 100, 100)])
def test_value_scales_at_the_ends_of_their_range(lead, early, late, count, dim, page):
    """Scores of later pages `lead` powers of two above those of the first 512 places, V scales 2^early and 2^late."""
    dev = require_gpu()
    c = make([count], [1300], 2, 1, dim, page, seed=40)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    c["k"][:] = 0
    for j, p in enumerate(c["table"][0, :-(-1300 // page)]):
        first = j * page < 512
        c["vs"][p], c["ks"][p] = 2.0 ** (early if first else late), 1.0 if first else lead
        if not first:
            c["k"][p, :, 5, 0] = code_of(1.0)
    scale = float(np.float32(np.log(2.0)))  # a score of 1 is a power of two
    for causal in (False, True):
        assert_weighted(attend(c, dev, causal, scale=scale), *reference(c, causal, scale))


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("count,length,heads,kv_heads,dim", [(1, 1300, 4, 2, 64), (1, 5000, 4, 2, 128), (40, 1300, 4, 2, 128),
                                                             (300, 1300, 4, 2, 64), (300, 1300, 4, 2, 128),
                                                             (1100, 2000, 64, 64, 128), (2000, 2000, 4, 4, 128)])
def test_equal_values_come_back_whatever_the_weights(count, length, heads, kv_heads, dim, page):
    """The weights of a row sum to one: of values that are all 1.5 (as 1.5 * 1 and as 3 * 0.5) the result is 1.5,
    with nothing but fp32 sums (2^-13 at these lengths) in between, and 2^-8 away from the next result."""
    dev = require_gpu()
    c = make([count], [length], heads, kv_heads, dim, page, seed=41)
    c["q"] *= 3
    for j, p in enumerate(c["table"][0, :-(-length // page)]):
        c["v"][p], c["vs"][p] = code_of(3.0 if j % 2 else 1.5), 0.5 if j % 2 else 1.0
    for causal in (False, True):
        got = attend(c, dev, causal)
        assert bool((got == 1.5).all()), float((got.float() - 1.5).abs().max())


def test_no_table_leaves_rows_of_no_request():
    dev = require_gpu()
    cache = fp8.Fp8KVCache(2, 2, device=dev)
    table = torch.empty((2, 0), dtype=torch.int32, device=dev)
    lengths, starts = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([4, 4], [2, 3, 6]))
    q = torch.ones((9, 4, 128), dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, 7.0)
    assert cache.attend(q, table, lengths, starts, out=out) is out
    assert not out[2:6].any() and bool((out[:2] == 7).all()) and bool((out[6:] == 7).all())


def at_odd_columns(x, dev, column):
    """x [tokens, heads, dim] as columns of a wider tensor, from this one on."""
    tokens, heads, dim = x.shape
    wide = torch.zeros((tokens, column + heads * dim + 3), dtype=x.dtype, device=dev)
    wide[:, column:column + heads * dim] = x.reshape(tokens, -1)
    return wide[:, column:column + heads * dim].unflatten(1, (heads, dim))


@pytest.mark.parametrize("tokens", [1, 2])
@pytest.mark.parametrize("heads", [1, 2])
@pytest.mark.parametrize("column", [0, 4, 8, 9])
def test_rows_at_any_address(column, heads, tokens):
    """A layer that works for a prompt works for its single-token steps: slices that begin anywhere."""
    dev = require_gpu()
    rng = torch.Generator().manual_seed(42)
    q, k, v = (torch.randn((tokens, heads, 128), generator=rng).to(torch.bfloat16) for _ in range(3))
    pos = torch.arange(3 * tokens, dtype=torch.int32, device=dev).view(tokens, 3)
    rope = fp8.RopeAxes(128, (16, 56, 56))
    whole = [x.to(dev) for x in (q, k, v)]
    odd = [at_odd_columns(x, dev, column) for x in (q, k, v)]
    for got, want in zip(rope(odd[0], odd[1], pos), rope(whole[0], whole[1], pos)):
        assert torch.equal(got, want)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=dev)
    lengths, starts = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([tokens], [0, tokens]))
    outs = []
    for x in (whole, odd):
        cache = fp8.Fp8KVCache(2, heads, device=dev)
        cache.append(x[1], x[2], table, lengths, starts)
        outs.append((cache.attend(x[0], table, lengths, starts), cache.k_codes[1, :, :tokens], cache.v_codes[1, :, :, :tokens],
                     cache.k_scale[1], cache.v_scale[1]))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_strides_of_single_rows_do_not_matter():
    """A dimension of size one may have any stride, of an input and of an output."""
    dev = require_gpu()
    rope = fp8.RopeAxes(64, (32, 32))
    pos = torch.tensor([[3, 5]], dtype=torch.int32, device=dev)
    x = torch.randn((1, 1, 64), device=dev).to(torch.bfloat16)
    want = rope(x, None, pos)[0]
    for token, head in ((1, 64), (64, 3), (0, 0), (7, 7)):
        out = torch.zeros(64, dtype=torch.bfloat16, device=dev).as_strided((1, 1, 64), (token, head, 1))
        got = rope(x.view(64).as_strided((1, 1, 64), (token, head, 1)), None, pos, q_out=out)[0]
        assert got is out and torch.equal(got, want)


def test_tables_whose_places_pass_64_bits_are_refused():
    dev = require_gpu()
    cache = fp8.Fp8KVCache(2, 2, device=dev)
    x = torch.ones((1, 2, 128), dtype=torch.bfloat16, device=dev)
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    lengths, starts = (torch.tensor(n, dtype=torch.int32, device=dev) for n in ([1], [0, 1]))
    rows = ctypes.byref(_lib.Rows(x.data_ptr(), 2, 256, 128))
    for pages in ((1 << 58) + 1, (1 << 62) + 1, (1 << 24) + 1):  # times 64 places
        assert _lib.lib().fp8_kv_append(cache._cache, 1, 1, rows, rows, table.data_ptr(), pages, lengths.data_ptr(),
                                        starts.data_ptr(), None) == _lib.ERR_BAD_SHAPE
        assert _lib.lib().fp8_kv_attend(cache._cache, 1, 1, rows, table.data_ptr(), pages, lengths.data_ptr(),
                                        starts.data_ptr(), 1.0, 0, x.data_ptr(), None, 0, None) == _lib.ERR_BAD_SHAPE
        assert cache.workspace_bytes(1, 1, 2, pages) == 0
    for refused in ((1 << 62, 1, 2, 9), (1, 1 << 62, 2, 9), (1, 1, 3, 9), (1, 1, 1 << 62, 9)):
        assert cache.workspace_bytes(*refused) == 0
    assert cache.workspace_bytes(1, 1, 2, 1 << 10) > 0


def test_parts_do_not_make_a_call_too_large():
    """Sizes of which a cut into parts would be more than a launch holds are served without."""
    dev = require_gpu()
    requests, tokens = 1170, (1 << 24) - 1
    cache = fp8.Fp8KVCache(1, 2, device=dev)
    row = torch.randn((1, 2, 128), device=dev).to(torch.bfloat16)
    starts, lengths = (torch.zeros(n, dtype=torch.int32, device=dev) for n in (requests + 1, requests))
    starts[-1] = lengths[-1] = 5  # the last request has five rows, the others none
    table = torch.full((requests, 308278), -1, dtype=torch.int32, device=dev)
    table[-1, 0] = 0
    five = row.expand(5, 2, 128)
    cache.append(five, five, table[-1:], lengths[-1:], starts[-2:])
    out = torch.empty((tokens, 2, 128), dtype=torch.bfloat16, device=dev)
    out[5:9] = 7.0
    assert cache.workspace_bytes(requests, tokens, 2, table.shape[1]) == 0
    cache.attend(row.expand(tokens, 2, 128), table, lengths, starts, out=out)
    assert torch.equal(out[:5], cache.attend(five, table[-1:], lengths[-1:], starts[-2:]))
    assert bool((out[5:9] == 7).all())


def test_calls_beyond_the_limits_are_refused():
    """On the host, whatever the addresses: more requests, or more workgroups, than the header allows."""
    dev = require_gpu()
    cache = fp8.Fp8KVCache(2, 2, device=dev)
    x = torch.ones((1, 2, 128), dtype=torch.bfloat16, device=dev)
    ints = torch.zeros(2, dtype=torch.int32, device=dev)
    lib, at = _lib.lib(), ints.data_ptr()

    def run(requests, tokens, heads):
        rows = ctypes.byref(_lib.Rows(x.data_ptr(), heads, 0, 0))
        return lib.fp8_kv_attend(cache._cache, requests, tokens, rows, at, 1, at, at, 1.0, 0, x.data_ptr(), None, 0, None)

    for requests, tokens, heads in ((_lib.MAX_REQUESTS + 1, 1, 2), (1, _lib.MAX_ROWS - 1, 65534), (1, 1 << 21, 2048)):
        assert run(requests, tokens, heads) == _lib.ERR_BAD_SHAPE
        assert cache.workspace_bytes(requests, tokens, heads, 1) == 0
    rows = ctypes.byref(_lib.Rows(x.data_ptr(), 2, 256, 128))
    assert lib.fp8_kv_append(cache._cache, _lib.MAX_REQUESTS + 1, 1, rows, rows, at, 1, at, at, None) == _lib.ERR_BAD_SHAPE


def test_a_workspace_is_dense():
    """Strided or broadcast elements are not as many bytes in a row."""
    dev = require_gpu()
    c = make([1], [4000], 2, 2, 128, 64, seed=44)
    cache, *batch = on_gpu(c, dev)
    need = cache.workspace_bytes(1, 1, 2, batch[0].shape[1])
    assert need > 0
    for ws in (torch.empty(1, dtype=torch.uint8, device=dev).expand(need), torch.empty(2 * need, dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            cache.attend(c["q"].to(dev), *batch, workspace=ws)


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("counts", [[1], [1, 1, 1], [20, 1, 33], [300, 1, 1, 7], [1, 1, 900, 1]])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_table_much_wider_than_the_lengths(dim, counts, page):
    """As a captured step holds it, and prompts beside single tokens: parts with nothing in them."""
    dev = require_gpu()
    c = make(counts, [n + 90 + 200 * i for i, n in enumerate(counts)], 4, 2, dim, page, seed=43)
    wide = np.full((len(counts), 700), -1, np.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide
    # some rows have a token of 0.95 of the weight: the whole term, 2^-7 of the weight
    for causal in (False, True):
        assert_weighted(attend(c, dev, causal), *reference(c, causal))


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("count,dim", FORMS + [(20, 128), (500, 128)])
@pytest.mark.parametrize("faint,size", [(-45, 110), (-35, 119), (-60, 60), (-60, -60), (-60, 0)])
def test_faint_tokens_where_strong_ones_hold_zero(faint, size, count, dim, page):
    """A column that the strongest token leaves at zero is made of tokens far below it, on places far away."""
    dev = require_gpu()
    c = make([count], [5000], 2, 1, dim, page, seed=45)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    c["k"][:], c["v"][:], c["ks"][:], c["vs"][:] = 0, 0, 1.0, 2.0 ** size
    for place, score, column in ((100, 100, 0), (2000, 100 + faint, 1), (4000, 100 + faint, 2)):
        p = c["table"][0, place // page]
        c["ks"][p] = score
        c["k"][p, :, place % page, 0] = code_of(1.0)
        c["v"][p, :, column, place % page] = code_of(1.0)
    scale = float(np.float32(np.log(2.0)))  # a score of 1 is a power of two
    got, (ref, weight) = attend(c, dev, scale=scale), reference(c, False, scale)
    assert_weighted(got, ref, weight)
    assert np.count_nonzero(bf16_out_to_f64(got)) == np.count_nonzero(ref) == 3 * 2 * count


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("count,dim", FORMS + [(20, 128), (500, 128)])
@pytest.mark.parametrize("seed", range(6))
def test_value_scales_anywhere_within_2_to_the_100(seed, count, dim, page):
    """Random scales and scores of all sizes. What stands 2^-70 below a row's largest column may be lost to fp32."""
    dev = require_gpu()
    rng = np.random.default_rng(46 + seed)
    c = make([count, 1], [1300, 900], 4, 2, dim, page, seed=47 + seed)
    least = [-100, -60, -30, -5, 10, 19][seed]
    c["vs"] = (2.0 ** rng.uniform(least, least + 100, c["vs"].shape)).astype(np.float32)
    c["q"] *= 2.0 ** (seed - 1)
    s = float(c["q"].double().abs().sum(-1).max()) * float(np.nanmax(c["ks"])) * 448 * dim ** -0.5
    for causal in (False, True):
        ref, weight = reference(c, causal)
        # scores of this size in fp32: 2^-16 of their terms' sum, as in the tests of large scores
        assert_weighted(attend(c, dev, causal), ref, weight, 2.0 ** -16 * s, 2.0 ** -70 * weight.max(-1, keepdims=True))


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("count,dim", FORMS + [(20, 128), (500, 128)])
@pytest.mark.parametrize("first", [512, 64])
def test_weights_below_a_bound_that_jumps(first, count, dim, page):
    """Tokens of tiny values whose weight, 2^3 of that of the tokens of large values behind them, is all in the
    denominator: the bound of the row rises by 2^127 in between."""
    dev = require_gpu()
    c = make([count], [1300], 2, 1, dim, page, seed=48)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    c["k"][:] = 0
    for j, p in enumerate(c["table"][0, :-(-1300 // page)]):
        if j * page < first:  # sets the bound of the row to 0
            c["vs"][p], c["ks"][p] = 2.0 ** -60, 60
            c["k"][p, :, :, 0] = code_of(1.0)
        else:
            late = j * page >= 1024
            c["vs"][p], c["ks"][p] = 2.0 ** (40 if late else -60), 87 if late else 90
            c["k"][p, :, 7, 0] = code_of(1.0)
    scale = float(np.float32(np.log(2.0)))
    assert_weighted(attend(c, dev, scale=scale), *reference(c, False, scale))
