"""Shared by the tests of the 4-bit paged cache: page tables, caches filled through the
library, and what the oracle says they hold."""
import numpy as np
import torch

from oracle import cache as ref
from scaled_dot_product_flash_gb300 import api

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def make_table(rng, lens, page, width=None, spare=2):
    """(table [B, width], number of pages): the pages each length needs, in random order, every
    other entry pointing outside the cache."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    width = max([1] + need) if width is None else width
    table = np.full((len(lens), width), -7, dtype=np.int32)
    order, at = rng.permutation(total), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table), total


def draw_rows(rng, shape, dtype, spread=1.0):
    return torch.from_numpy(spread * rng.standard_normal(shape)).to(TYPES[dtype])


def dirty_cache(pages, heads, page, D, dtype):
    """A cache whose every byte is 0xff: codes 15, scales and zeros NaN."""
    cache = api.cache_empty(pages, heads, page, D, TYPES[dtype])
    cache.view(torch.uint8).fill_(255)
    return cache


def held(x, dtype):
    """What the cache holds of fp64 rows x, in fp64."""
    return ref.values(*ref.quantise(x, TYPES[dtype]))
