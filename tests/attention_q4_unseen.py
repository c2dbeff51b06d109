"""What the tests of unseen slots of 4-bit pools share."""
import numpy as np
import torch

from tests import attention_q4_ref as q4

# scale, low, codes of a group at the ends of f16: finite, and 15 times such a scale is none
ENDS = [(0x7BFF, 0x0000, 0xFF), (0x7BFF, 0x7BFF, 0xFF), (0xFBFF, 0xFBFF, 0xF0)]


def vector(D, scale, low, codes):
    """A head vector all of whose groups are such."""
    pair = np.array([scale, low] * (D // 32), np.uint16).view(np.uint8)
    return torch.from_numpy(np.concatenate([np.full(D // 2, codes, np.uint8), pair]))


def small_values(D, by=-10):
    """An edit_bytes that multiplies the values by a power of two."""
    def edit(b):
        pair = b[:, 1, :, D // 2:].view(np.float16)
        pair[:] = pair * np.float16(2.0 ** by)
    return edit


def no_token(c):
    """The pool's head vectors, and which of them belong to no token (pools without gaps)."""
    v = c.pool.view(-1, c.D // 8 * 5)
    return v, (v == 0xFF).all(1)


def slots(c, positions):
    """The slots of positions of the prefix or of request 0."""
    return [int(c.prefix_pages[j // c.page] if j < c.prefix else c.tables[0, j // c.page]) * c.page + j % c.page
            for j in positions]


def run(c):
    return [x.clone() for x in q4.Run(c).call().results()]
