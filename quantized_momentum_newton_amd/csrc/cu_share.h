// How many workgroups of a launch a CU takes (host only).
#pragma once

namespace qm {
namespace {

// LDS bytes of a launch that uses none: a workgroup that claims a share of a
// CU's 160 KiB keeps the number of workgroups on the CU down.  A stream of many
// tensors runs faster with fewer waves than fit: about as many as hold 40 to
// 80 KiB of loads in flight on a CU (more of them only spread the accesses in
// flight over more of memory).  The shares below were measured against each
// other on the same buffers, call by call in turn.  LDS is given out in units
// of 1280 bytes.
constexpr unsigned wgs_per_cu(unsigned n) { return (160u << 10) / n / 1280 * 1280; }

}  // namespace
}  // namespace qm
