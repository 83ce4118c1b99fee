// Host-side pieces the collectives and the block operators share.
#pragma once

#include <string>

namespace ringar {

// Text behind ringar_last_error() (one per thread).
std::string& last_error_text();

// Frees every workspace of the block operators (ringar_release).  Returns
// false if a HIP call failed; the text is then in last_error_text().
bool release_workspaces();

}  // namespace ringar
