"""CPU test of the rotary table's scaling by parts, between its two ends."""
import math

import pytest
import torch

import expert_layer_gb300 as moe


@pytest.mark.parametrize("rot,base,factor,trained,fast,slow", [
    (64, 10000.0, 8.0, 1024, 32.0, 1.0), (128, 1e6, 4.0, 4096, 32.0, 1.0), (128, 500000.0, 16.0, 8192, 16.0, 2.0),
    (32, 10000.0, 1.0, 2048, 32.0, 1.0)])
def test_by_parts_blends_linearly(rot, base, factor, trained, fast, slow):
    """Pair i turns trained * base^(-2i/rot) / (2 pi) times over the trained length.  Up to the whole index at or
    below where that is `fast` frequencies stay, from the one at or above where it is `slow` they are divided, and
    in between the share that stays falls linearly in i."""
    def index(turns):                      # solves turns = trained base^(-2i/rot) / (2 pi) for i
        return rot / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)
    low, high = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
    table = moe.rope_table(64, rot, base=base, scaling="by_parts", factor=factor, original_max_pos=trained,
                           beta_fast=fast, beta_slow=slow, device="cpu")
    mul, middle = 0.1 * math.log(factor) + 1, 0
    for i in range(rot // 2):
        stay = 1.0 if i <= low else 0.0 if i >= high else 1 - (i - low) / (high - low)
        middle += 0 < stay < 1
        f = base ** (-2 * i / rot) * (stay + (1 - stay) / factor)
        for p in (1, 17, 63):
            # fp32 of values up to mul, angles in fp64
            assert abs(float(table[p, i]) - mul * math.cos(p * f)) <= mul * 2.0 ** -23
            assert abs(float(table[p, rot // 2 + i]) - mul * math.sin(p * f)) <= mul * 2.0 ** -23
    assert middle >= 3
