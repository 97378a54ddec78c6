"""Prompt writes into the 8-bit cache while another stream builds the angle tables of
their theta (GPU; a process of its own, where no table has been built)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from _gpu_util import binding, cuda_or_skip
from _kv8_util import D, as_pool, bits, put_block, rotated
from _longctx_util import HKV, P
from test_gpu_kv8 import bf16, err_of, i32, oracle_bits, same

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
# before the tables' end, across it and past it, whole blocks and parts of them
STARTS, COUNT, COPIES, WRITES = (0, 2040, 5000), 100, 40, 40
PAGES = COUNT // P + 2                                # of a sequence


def expected(k, v, theta):
    """Codes and scales [3 * PAGES] of the three sequences, in 64 bits."""
    codes = np.zeros((len(STARTS) * PAGES, 2, HKV, P, D), np.uint8)
    scales = np.full(codes.shape[:3], 100, np.uint8)
    for i, start in enumerate(STARTS):
        rows = slice(i * COUNT, (i + 1) * COUNT)
        both = rotated(k[rows], range(start, start + COUNT), theta), oracle.bf16_to_f64(v[rows])
        for page0 in range(start // P * P, start + COUNT, P):
            a, z = max(start, page0), min(start + COUNT, page0 + P)
            page = i * PAGES + page0 // P - start // P
            for kv, x in enumerate(both):
                for h in range(HKV):
                    codes[page, kv, h], scales[page, kv, h] = put_block(
                        codes[page, kv, h], scales[page, kv, h], a - page0,
                        x[a - start:z - start, h], "int8")
    return codes, scales


def write_beside_a_table(theta, cycles, seed):
    """WRITES writes on one stream, a CTA to a page or two, while another stream sleeps,
    builds theta's tables and writes too; all as the definition says."""
    dev, b = torch.device("cuda", 0), binding()
    rng = np.random.default_rng(seed)
    few, batch = len(STARTS), len(STARTS) * COPIES
    k, v = (oracle_bits(rng.standard_normal((few * COUNT, HKV, D)).astype(np.float32))
            for _ in range(2))
    kk, vv = (bf16(np.tile(x, (COPIES, 1, 1)), dev) for x in (k, v))
    bt = np.full((batch, max(STARTS) // P + PAGES), -1, np.int32)
    for s in range(batch):
        first = STARTS[s % few] // P
        bt[s, first:first + PAGES] = np.arange(s * PAGES, (s + 1) * PAGES)
    bt, off = i32(bt, dev), i32(np.arange(batch + 1) * COUNT, dev)
    starts = i32(STARTS * COPIES, dev)
    pools = [(torch.zeros((batch * PAGES, 2, HKV, P, D), dtype=torch.int8, device=dev),
              torch.full((batch * PAGES, 2, HKV), 100, dtype=torch.uint8, device=dev))
             for _ in range(WRITES + 1)]
    err = err_of(dev)
    builder, writer = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(builder):
        torch.cuda._sleep(cycles)
    for i, (pool, sc) in enumerate(pools):
        b.kv8_write_prefill(kk, vv, off, starts, pool, sc, bt, rope_theta=theta, dev_err=err,
                            stream=builder if i == 0 else writer)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    codes, scales = expected(k, v, theta)
    for i, (pool, sc) in enumerate(pools):
        same(bits(sc), np.tile(scales, (COPIES, 1, 1)), f"write {i}: scales")
        same(bits(pool), np.tile(codes, (COPIES, 1, 1, 1, 1)), f"write {i}: codes")


def main():
    # (a device holds four tables)
    for i, (theta, cycles) in enumerate([(1e4, 200_000), (5e5, 600_000), (1e6, 1_200_000),
                                         (2e4, 2_000_000)]):
        write_beside_a_table(theta, cycles, i)


def test_writes_beside_a_table_that_is_built():
    cuda_or_skip()
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(HERE), HERE]))
    r = subprocess.run([sys.executable, "-c", "import test_gpu_kv8_tables as t; t.main()"],
                       cwd=HERE, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
