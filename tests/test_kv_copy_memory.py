"""What the page copy refuses of memory that caches and bounds share: nothing is
written twice, and no page of it is both read and written.  (No call here
launches anything: where nothing is refused, no pair has tokens.)"""
import pytest

import heterogeneous_adapter_batching_amd as hl
from test_kv_pages import bounds, copy, kv

MB = 1 << 20


def cache(i, **change):
    """A quantised cache of memory of its own, number i."""
    f = dict(k=(8 * i + 1) * MB, v=(8 * i + 2) * MB, k_scale=(8 * i + 3) * MB, v_scale=(8 * i + 4) * MB,
             dtype=hl.LORA_KV_E4M3)
    f.update(change)
    return kv(**f)


def summary(i, **change):
    f = dict(codes=(8 * i + 5) * MB, exps=(8 * i + 6) * MB)
    f.update(change)
    return bounds(**f)


ONE, TWO, THREE, FOUR = (cache(i) for i in range(4))
B = [summary(i) for i in range(4)]


def none(**args):
    """A copy of no tokens of one pair."""
    return copy([1], [2], [0], **args)


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
@pytest.mark.parametrize("other", ["k", "v", "k_scale", "v_scale"])
def test_destinations_that_share_a_tensor(name, other):
    to = [THREE, cache(3, **{name: getattr(THREE, other)})]
    assert none(caches=[ONE, TWO], to=to) == hl.LORA_EINVAL
    assert none(caches=[ONE, TWO], to=to[::-1]) == hl.LORA_EINVAL
    assert none(caches=[ONE, TWO], to=[THREE, FOUR]) == hl.LORA_OK


@pytest.mark.parametrize("name", ["codes", "exps"])
@pytest.mark.parametrize("other", ["codes", "exps"])
def test_destinations_that_share_bounds(name, other):
    args = dict(caches=[ONE, TWO], to=[THREE, FOUR], b=B[:2])
    assert none(to_b=[B[2], summary(3, **{name: getattr(B[2], other)})], **args) == hl.LORA_EINVAL
    assert none(to_b=B[2:], **args) == hl.LORA_OK


@pytest.mark.parametrize("names", [("k", "v"), ("k_scale", "v_scale")])
def test_keys_and_values_of_one_memory(names):
    """One tensor for keys and values is copied from such a one, not from two."""
    def alike(i):
        c = cache(i)
        return cache(i, **{names[1]: getattr(c, names[0])})
    assert none(caches=[ONE], to=[alike(2)]) == hl.LORA_EINVAL
    assert none(caches=[ONE, TWO], to=[FOUR, alike(2)]) == hl.LORA_EINVAL
    assert none(caches=[alike(0)], to=[alike(2)]) == hl.LORA_OK
    assert none(caches=[alike(0)], to=[THREE]) == hl.LORA_OK  # to two of their own
    assert none(caches=[alike(0)]) == hl.LORA_OK


def test_one_memory_in_two_layouts():
    """Within caches, pages of one are not pages of the other."""
    other = cache(0, page_stride=8192)
    assert none(caches=[ONE, ONE]) == hl.LORA_OK
    assert none(caches=[ONE, other]) == hl.LORA_EINVAL
    assert none(caches=[ONE, TWO, other]) == hl.LORA_EINVAL
    assert none(caches=[ONE, cache(1, v=ONE.k, token_stride=256)]) == hl.LORA_EINVAL


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
@pytest.mark.parametrize("other", ["k", "v", "k_scale", "v_scale"])
def test_a_tensor_that_is_read_and_written(name, other):
    to = [cache(2, **{name: getattr(ONE, other)})]
    assert copy([1, 2], [2, 3], [0, 0], caches=[ONE], to=to) == hl.LORA_EINVAL
    assert copy([1], [1], [0], caches=[ONE], to=to) == hl.LORA_EINVAL
    assert copy([1, 1], [2, 3], [0, 0], caches=[ONE], to=to) == hl.LORA_OK


@pytest.mark.parametrize("name", ["codes", "exps"])
def test_bounds_that_are_read_and_written(name):
    """Only whole pages have bounds that move: of the others any may be read and written."""
    to_b = [summary(2, **{name: getattr(B[0], name)})]
    args = dict(caches=[ONE], to=[THREE], b=B[:1], to_b=to_b)
    for tokens in (None, [16, 16], [16, 16, 0]):
        src, dst = [1, 2, 5][:len(tokens or "12")], [2, 3, 6][:len(tokens or "12")]
        assert copy(src, dst, tokens, **args) == hl.LORA_EINVAL
    assert copy([2, 1], [3, 2], [16, 16], **args) == hl.LORA_EINVAL
    assert copy([1, 2], [2, 3], [0, 0], **args) == hl.LORA_OK
    crosswise = dict(caches=[ONE, TWO], to=[THREE, FOUR], b=B[:2],
                     to_b=[summary(2, **{name: getattr(B[1], name)}), summary(3, **{name: getattr(B[0], name)})])
    for src, dst in (([1, 2], [2, 3]), ([1], [1])):  # each page's bounds from the other cache
        assert copy(src, dst, None, **crosswise) == hl.LORA_EINVAL
        assert copy(src, dst, [0] * len(src), **crosswise) == hl.LORA_OK


@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("other", ["k", "v"])
def test_one_memory_read_in_one_layout_and_written_in_another(name, other):
    """Page numbers say nothing about what overlaps."""
    for change in (dict(page_stride=8192), dict(head_stride=4096), dict(token_stride=256)):
        assert none(caches=[ONE], to=[cache(2, **{name: getattr(ONE, other)}, **change)]) == hl.LORA_EINVAL
        assert none(caches=[ONE, TWO], to=[cache(2, **change), cache(3, **{name: getattr(ONE, other)}, **change)]) == hl.LORA_EINVAL
        assert none(caches=[ONE], to=[cache(2, **change)]) == hl.LORA_OK
    assert none(caches=[ONE], to=[cache(2, **{name: getattr(ONE, other)})]) == hl.LORA_OK
