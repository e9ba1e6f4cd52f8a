"""The benchmark's JSON line stays short enough to be kept whole."""
import importlib.util
import json
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("bench", os.path.join(ROOT, "bench.py"))
bench = importlib.util.module_from_spec(spec)
spec.loader.exec_module(bench)


def test_the_line_is_short_and_keeps_its_keys():
    row = dict(shape="w8a8_int8_prefill_residual", quant="w8a8_int8", M=32768, N=12288, K=14336,
               variant="tile bm=256 bn=256 wm=2 wn=4 group=4 streamk=1 stages=3", us=12345.678,
               TBps=1.2345, TFLOPs=1234.567, hbm_frac=0.1234, mfma_frac=0.1234, bound="hbm",
               kernels_per_call=1, roof_frac=0.1234, of_stream_ceiling=0.1234)
    size = dict(MiB=96, bytes=1 << 27, copies=32, us=18.123, TBps=5.1234, hbm_frac=0.6789, grid=2048,
                unroll=8, all_us={f"{g}x{u}": 12.345 for g in (512, 1024, 2048, 4096) for u in (4, 8, 16)})
    keys = ("metric value unit n_gpus steps warmup ms_per_step higher_is_better scaling vs_baseline "
            "dtype data config").split()
    out = dict({k: "x" * 20 for k in keys}, shapes=[row] * 60, hbm_stream_ceiling=[size] * 4,
               roofline={"x": "y" * 350}, per_M=[{"x": "y" * 180}] * 7, cpu_baseline={"x": "y" * 200})
    line = bench.json_line(out)
    assert "\n" not in line and len(line) < 12000, len(line)
    got = json.loads(line)
    assert all(got[k] == out[k] for k in keys) and len(got["shapes"]) == 60
    assert got["shapes"][0]["us"] == row["us"] and got["hbm_stream_ceiling"][0]["TBps"] == size["TBps"]
    assert json.loads(bench.json_line(dict(out, shapes=None)))["shapes"] is None
