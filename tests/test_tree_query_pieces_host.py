"""What the e4m3 pieces of a 2-byte query row leave of its elements, over all
significands and magnitudes, against the accuracy that the header promises."""
import os
import re

import pytest
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pafp8.h")


def e4m3(x):
    return x.to(torch.float8_e4m3fn).float()


def left_over(pieces, dtype):
    """(elements scaled so that the row's largest lies in [128, 256), what the
    pieces leave): every element of the type up to 256."""
    bits = torch.arange(0x7C00 if dtype is torch.float16 else 0x7F80, dtype=torch.int32).to(torch.int16).view(dtype)
    x = bits.float()
    if dtype is torch.float16:  # a scale brings rows of small values up: the significands of all magnitudes
        x = torch.cat([x * 2.0 ** -s for s in (0, 8, 16, 24)])
    x = x[(x > 0) & (x < 256)]
    h = x.half()                # in f16, as the kernel
    rest = h.clone()
    for _ in range(pieces):
        rest = (rest - e4m3(rest.float()).half())
    return x, (x - h.float() + rest.float()).abs()


@pytest.mark.parametrize("dtype,pieces", [(torch.bfloat16, 2), (torch.float16, 3)])
def test_the_header_states_what_the_pieces_leave(dtype, pieces):
    with open(HEADER) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    m = re.search(r"multiplied exactly but for elements below 2\^-(\d+) \(bf16\) or 2\^-(\d+) \(f16\) of its row's largest "
                  r"magnitude, which lose 2\^-(\d+) of it at most", text)
    assert m, "the header states no accuracy of a 2-byte query over an fp8 cache"
    below = 2.0 ** -int(m.group(1 if dtype is torch.bfloat16 else 2))
    loss = 2.0 ** -int(m.group(3))
    x, rest = left_over(pieces, dtype)
    # The row's largest may be as small as 128 (it is in [128, 256)).
    assert float(rest.max()) <= 128 * loss
    assert float(rest[x >= 128 * below].max()) == 0.0
    # and neither could be stated half as large
    assert float(rest.max()) > 64 * loss and float(rest[x >= 64 * below].max()) > 0.0
