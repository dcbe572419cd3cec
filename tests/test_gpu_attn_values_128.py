"""GPU: the cases of test_gpu_attn_values with heads of 128 instead of 64."""

import pytest

import test_gpu_attn_values as values

pytestmark = pytest.mark.gpu

CASES = ["rows_without_weight_are_zeros_whatever_their_values", "infinite_queries_do_not_reach_keys_that_are_not_valid",
         "infinite_values_in_valid_places", "flat_tail_far_below_one_leading_key", "scores_up_to_the_largest",
         "scales_at_the_ends_of_their_range"]


@pytest.fixture(autouse=True)
def heads_of_128(monkeypatch):
    monkeypatch.setattr(values, "DIM", 128)


@pytest.mark.parametrize("form,dt", values.ALL)
@pytest.mark.parametrize("case", CASES)
def test_heads_of_128(case, form, dt):
    getattr(values, "test_" + case)(form, dt)


@pytest.mark.parametrize("form,dt", values.ALL)
def test_infinite_values_of_small_weight(form, dt):
    values._infinite_values_of_small_weight(form, dt)


@pytest.mark.parametrize("form", ["paged", "paged-short", "paged-cut", "token", "rows"])
def test_few_rows_keep_more_than_float16_weights(form):
    values.test_few_rows_keep_more_than_float16_weights(form)
