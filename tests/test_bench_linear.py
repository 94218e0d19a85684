"""The benchmark times the NVFP4 linear, whose FP4 GEMM has multicast loads, on one GPU only."""
import argparse

import pytest

import bench


def test_linear_is_timed_on_one_gpu_only():
    args = argparse.Namespace(skip_linear=False)
    assert bench.with_linear(args, 1)
    assert not any(bench.with_linear(args, ws) for ws in (2, 4, 8))
    assert not bench.with_linear(argparse.Namespace(skip_linear=True), 1)


@pytest.mark.parametrize("gpus,world", [("2", "1"), ("1", "2")])
def test_linear_only_refuses_several_gpus(gpus, world, monkeypatch):
    monkeypatch.setenv("WORLD_SIZE", world)
    with pytest.raises(SystemExit):
        bench.main(["--linear-only", "--gpus", gpus, "--warmup", "3"])
