"""The committed record of the attention kernels' DRAM traffic: it was taken on
the sources that are here, so that the bench line has its figure, and what
voids it is a change of those kernels, not of other calls' declarations."""
import os
import shutil

import bench


def test_the_record_is_of_these_sources():
    for role in ("fwd", "bwd"):
        rec = bench.traffic_record(f"heavy_tailed:{role}")
        assert rec is not None, f"profiles/traffic.json: take the {role} capture again ({bench.kernel_sources_sha(role)})"
        assert rec["dram_bytes_per_token"] > 0 and rec["capture_tokens"] > 0


def test_what_voids_it(monkeypatch, tmp_path):
    csrc = os.path.join("hstu_jagged_attention_02_gb300", "csrc")
    shutil.copytree(os.path.join(bench.ROOT, csrc), tmp_path / csrc)
    shutil.copytree(os.path.join(bench.ROOT, "include"), tmp_path / "include")
    now = {r: bench.kernel_sources_sha(r) for r in ("fwd", "bwd")}
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert {r: bench.kernel_sources_sha(r) for r in now} == now
    header, unit = tmp_path / "include" / "hstu_attn.h", tmp_path / csrc / "hstu_tc_fwd.cu"
    text = header.read_text()
    header.write_text(text.replace("#ifdef __cplusplus\n}", "int hstu_another_call(int x);\n#ifdef __cplusplus\n}"))
    assert header.read_text() != text
    assert {r: bench.kernel_sources_sha(r) for r in now} == now      # another call
    header.write_text(text.replace("#define HSTU_FLAG_U_FP32 (1u << 2)", "#define HSTU_FLAG_U_FP32 (1u << 9)"))
    assert all(bench.kernel_sources_sha(r) != now[r] for r in now)   # a flag that the kernels read
    header.write_text(text)
    unit.write_text(unit.read_text() + "\nstatic int more;\n")
    assert bench.kernel_sources_sha("fwd") != now["fwd"] and bench.kernel_sources_sha("bwd") == now["bwd"]
